// Root-mean-square norm with the residual's addition, its result kept in 16 or
// 32 bits or written in the 8-bit forms that the products read, and its
// gradient.
//
//   h = x + residual,  rstd = 1 / sqrt(mean(h^2) + eps),  y = h rstd w
//   FP8:  per row and 128 columns s = max(amax |y|, 1e-12) / 448, codes E4M3(y / s)
//   INT8: per row s = max(amax |y|, 1e-12) / 127, codes rint(y / s)
// Everything between the loads and the stores is FP32: h and y are rounded once
// each, and y / s is taken from the unrounded h (y / s = (h w) (rstd / s)).
// amax |h w| needs no rstd, so the row's sum of squares and its largest
// magnitude are reduced together: one exchange between the warps per row.
//
// gradient, with g = d_y w:
//   d_x = rstd g - h rstd^3 mean(g h) (+ d_h),  d_w = sum over rows of d_y h rstd
//
// HBM-bound: every row is read once and stays in registers, 16 lanes per block
// of 128 columns, 8 columns per lane (Piece); `group` threads hold a row, kC
// pieces each.  What registers can hold in flight (32 KB per SM) is too little for
// HBM, so where there are many aligned rows they come through a ring in shared
// memory, filled by bulk copies some rows ahead.
#include <algorithm>

#include "common.cuh"
#include "elem.cuh"
#include "internal.h"

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
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int at = l + 16 * i;
        if constexpr (sizeof(T) == 2)
          w[i] = at < cols ? reinterpret_cast<const unsigned short*>(p)[at] : 0u;
        else
          w[i] = at < cols ? __float_as_uint(p[at]) : 0u;
      }
    }
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
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (l + 16 * i < cols) p[l + 16 * i] = (uint8_t)((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
    }
  }
};

__device__ __forceinline__ uint2 e4m3x8(const float (&v)[8], float f) {
  return make_uint2(e4m3x2(v[0] * f, v[1] * f) | e4m3x2(v[2] * f, v[3] * f) << 16,
                    e4m3x2(v[4] * f, v[5] * f) | e4m3x2(v[6] * f, v[7] * f) << 16);
}

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
__device__ __forceinline__ void load_weights(const void* w, bool w32, int64_t c, int l, int cols, float (&f)[8]) {
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

// (sum, largest) over the `group` threads that hold a row, in every one of them.
// Groups of more than a warp are whole warps of a block that comes here together;
// buf alternates between two buffers from row to row, so that one barrier per row
// is enough.
struct Exchange {
  float2 part[2][32];
};
template <bool kTop>
__device__ __forceinline__ float2 group_reduce(float sum, float top, int group, Exchange& ex, int buf) {
  const int width = min(group, 32);
  for (int o = width / 2; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (kTop) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  }
  if (group > 32) {
    const int lane = threadIdx.x & 31, warps = group >> 5, first = (threadIdx.x >> 5) / warps * warps;
    if (lane == 0) ex.part[buf][threadIdx.x >> 5] = make_float2(sum, top);
    __syncthreads();
    const float2 v = lane < warps ? ex.part[buf][first + lane] : make_float2(0.f, 0.f);
    sum = v.x, top = v.y;
    for (int o = warps > 8 ? 16 : 4; o > 0; o >>= 1) {
      sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (kTop) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
    sum = __shfl_sync(0xffffffffu, sum, 0);
    if (kTop) top = __shfl_sync(0xffffffffu, top, 0);
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
  __device__ __forceinline__ int64_t at(int i) const { return (int64_t)block(i) * 128; }
  __device__ __forceinline__ int cols(int i, int64_t H) const { return (int)min((int64_t)128, H - at(i)); }
};

// A row of h = x + residual in v: reduced, scaled by the weights and written.
template <typename T, bool kVec, int kC, int kForm, typename Weights, typename AfterReduce>
__device__ __forceinline__ void norm_row(const NormArgs& a, const Place& pl, int64_t row, bool live, float (&v)[kC][8], Exchange& ex,
                                         int buf, int* status, Weights&& weights, AfterReduce&& after_reduce) {
  using P = Piece<T, kVec>;
  auto cols = [&](int i) { return live ? pl.cols(i, a.H) : 0; };
  float sum = 0.f, top = 0.f;
#pragma unroll
  for (int i = 0; i < kC; ++i) {
    if (a.h) P::store(static_cast<T*>(a.h) + row * a.H + pl.at(i), pl.l, cols(i), v[i]);
    float w[8];
    weights(i, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      sum = fmaf(v[i][j], v[i][j], sum);
      v[i][j] *= w[j];
      if (kForm == Q4_NORM_INT8) top = fmaxf(top, fabsf(v[i][j]));
    }
  }
  const float2 r = group_reduce<kForm == Q4_NORM_INT8>(sum, top, pl.group, ex, buf);
  after_reduce();
  const float rstd = __frsqrt_rn(r.x / (float)a.H + a.eps);
  if (pl.t == 0 && live) {
    if (a.rstd) a.rstd[row] = rstd;
    if (nonfinite(r.x)) latch_status(status, Q4_ERR_NONFINITE);
  }
  // the codes' factor rstd / s may be off by 2 ulp, as rstd may
  if constexpr (kForm == Q4_NORM_INT8) {
    const float s = fmaxf(r.y * rstd, 1e-12f) * (1.f / 127.f);
    if (pl.t == 0 && live) {
      a.scales[row] = s;
      if (nonfinite(s)) latch_status(status, Q4_ERR_NONFINITE);
    }
    const float f = __fdividef(rstd, s);
#pragma unroll
    for (int i = 0; i < kC; ++i) P::store_codes(a.codes + row * a.H + pl.at(i), pl.l, cols(i), int8x8(v[i], f));
  }
  if constexpr (kForm == Q4_NORM_FP8) {
    const int blocks = (int)((a.H + 127) / 128);
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      float m = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[i][j]));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float s = fmaxf(m * rstd, 1e-12f) * (1.f / 448.f);
      P::store_codes(a.codes + row * a.H + pl.at(i), pl.l, cols(i), e4m3x8(v[i], __fdividef(rstd, s)));
      if (pl.l == 0 && cols(i) > 0) {
        a.scales[row * blocks + pl.block(i)] = s;
        if (nonfinite(s)) latch_status(status, Q4_ERR_NONFINITE);
      }
    }
  }
  if (a.y) {
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = v[i][j] * rstd;
      P::store(static_cast<T*>(a.y) + row * a.H + pl.at(i), pl.l, cols(i), y);
    }
  }
}

// Rows straight from global memory: few rows, or rows that 128-bit accesses do not
// fit (kVec false).
template <typename T, bool kVec, int kC, int kForm>
__global__ void __launch_bounds__(max_threads(kC))
    norm_kernel(const NormArgs a, int group, int* status) {
  pdl_wait();
  using P = Piece<T, kVec>;
  __shared__ Exchange ex;
  const Place pl(group);
  auto weights = [&](int i, float (&f)[8]) {
    load_weights<T, kVec>(a.weight, a.w_fp32, pl.at(i), pl.l, pl.cols(i, a.H), f);
  };
  int buf = 0;
  for (int64_t base = (int64_t)blockIdx.x * pl.per_block; base < a.rows; base += (int64_t)gridDim.x * pl.per_block, buf ^= 1) {
    const int64_t row = base + pl.sub;
    const bool live = row < a.rows;
    float v[kC][8];
    {
      P px[kC], pr[kC];
#pragma unroll
      for (int i = 0; i < kC; ++i)
        px[i].load(static_cast<const T*>(a.x) + row * a.ldx + pl.at(i), pl.l, live ? pl.cols(i, a.H) : 0);
      if (a.residual) {
#pragma unroll
        for (int i = 0; i < kC; ++i)
          pr[i].load(static_cast<const T*>(a.residual) + row * a.ld_residual + pl.at(i), pl.l, live ? pl.cols(i, a.H) : 0);
      }
#pragma unroll
      for (int i = 0; i < kC; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = a.residual ? px[i].at(j) + pr[i].at(j) : px[i].at(j);
    }
    norm_row<T, kVec, kC, kForm>(a, pl, row, live, v, ex, buf, status, weights, [] {});
  }
}

// ------------------------------------------------------------------ rows through shared memory
constexpr int kMaxRing = 8;
// A ring of stages, each the block's next per_block rows of up to three matrices.
struct Ring {
  uint64_t full[kMaxRing];
  int abort;
};
struct RingArgs {
  int stages;
  uint32_t stage_bytes, row_bytes;
  KernelCtl ctl;
};

__device__ __forceinline__ void ring_init(Ring& ring, const RingArgs& r) {
  if (threadIdx.x == 0) {
    for (int s = 0; s < r.stages; ++s) mbar_init(smem_u32(&ring.full[s]), 1);
    ring.abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
}

// One thread: rows base .. of the matrices into stage s.
template <int kMats>
__device__ __forceinline__ void ring_fill(Ring& ring, const RingArgs& r, uint32_t smem, int s, const void* const (&mat)[kMats],
                                          const int64_t (&pitch)[kMats], int64_t base, int64_t rows, int per_block) {
  const int n = (int)min((int64_t)per_block, rows - base);
  if (n <= 0) return;
  int mats = 0;
  for (int m = 0; m < kMats; ++m) mats += mat[m] != nullptr;
  const uint32_t bar = smem_u32(&ring.full[s]);
  mbar_arrive_expect_tx(bar, (uint32_t)(mats * n) * r.row_bytes);
  uint32_t dst = smem + s * r.stage_bytes;
  for (int m = 0; m < kMats; ++m) {
    if (!mat[m]) continue;
    const uint8_t* src = static_cast<const uint8_t*>(mat[m]) + base * pitch[m];
    if (pitch[m] == r.row_bytes)
      bulk_load(dst, src, (uint32_t)n * r.row_bytes, bar);
    else
      for (int i = 0; i < n; ++i) bulk_load(dst + i * r.row_bytes, src + i * pitch[m], r.row_bytes, bar);
    dst += (uint32_t)per_block * r.row_bytes;
  }
}

template <typename T, int kC, int kForm>
__global__ void __launch_bounds__(512, 1) norm_ring_kernel(const NormArgs a, int group, const RingArgs r) {
  extern __shared__ __align__(128) uint8_t stage_smem[];
  using P = Piece<T, true>;
  __shared__ Ring ring;
  __shared__ Exchange ex;
  ring_init(ring, r);
  pdl_wait();
  const Place pl(group);
  const void* const mat[2] = {a.x, a.residual};
  const int64_t pitch[2] = {a.ldx * (int64_t)sizeof(T), a.ld_residual * (int64_t)sizeof(T)};
  const int64_t step = (int64_t)gridDim.x * pl.per_block, base0 = (int64_t)blockIdx.x * pl.per_block;
  if (threadIdx.x == 0)
    for (int s = 0; s < r.stages; ++s) ring_fill(ring, r, smem_u32(stage_smem), s, mat, pitch, base0 + s * step, a.rows, pl.per_block);
  float w[kC][8];
#pragma unroll
  for (int i = 0; i < kC; ++i) load_weights<T, true>(a.weight, a.w_fp32, pl.at(i), pl.l, pl.cols(i, a.H), w[i]);
  int stage = 0, buf = 0;
  uint32_t phase = 0;
  for (int64_t base = base0; base < a.rows; base += step, buf ^= 1) {
    const int64_t row = base + pl.sub;
    const bool live = row < a.rows;
    mbar_wait(smem_u32(&ring.full[stage]), phase, r.ctl, &ring.abort);
    const T* x = reinterpret_cast<const T*>(stage_smem + stage * r.stage_bytes + pl.sub * r.row_bytes);
    const T* res = reinterpret_cast<const T*>(reinterpret_cast<const uint8_t*>(x) + pl.per_block * r.row_bytes);
    float v[kC][8];
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      P px;
      px.load(x + pl.at(i), pl.l, live ? pl.cols(i, a.H) : 0);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = px.at(j);
      if (a.residual) {
        P pr;
        pr.load(res + pl.at(i), pl.l, live ? pl.cols(i, a.H) : 0);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] += pr.at(j);
      }
    }
    norm_row<T, true, kC, kForm>(
        a, pl, row, live, v, ex, buf, r.ctl.status,
        [&](int i, float (&f)[8]) {
#pragma unroll
          for (int j = 0; j < 8; ++j) f[j] = w[i][j];
        },
        [&] {  // every thread has read the stage: the next rows may come
          if (pl.group <= 32) __syncthreads();
          if (threadIdx.x == 0)
            ring_fill(ring, r, smem_u32(stage_smem), stage, mat, pitch, base + r.stages * step, a.rows, pl.per_block);
        });
    if (++stage == r.stages) stage = 0, phase ^= 1;
  }
}

// ------------------------------------------------------------------ gradient
// Each block of threads takes every gridDim.x-th row (or as many rows as it has
// groups) and adds its rows' part of d_w up in registers, columns fixed to
// threads; the blocks' sums go to the workspace and are added in their order by
// a second kernel, so that results do not depend on timing.

// The block's part of d_w: the groups' sums one after another.
template <bool kVec, int kC>
__device__ __forceinline__ void store_partial(const NormBackwardArgs& a, const Place& pl, const float (&acc)[kC][8]) {
  if (!a.partial) return;
  float* out = a.partial + (int64_t)blockIdx.x * a.H;
  for (int s = 0; s < pl.per_block; ++s) {
    if (s) __syncthreads();
    if (pl.sub != s) continue;
#pragma unroll
    for (int i = 0; i < kC; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int c = kVec ? 8 * pl.l + j : pl.l + 16 * j;
        if (c < pl.cols(i, a.H)) out[pl.at(i) + c] = s ? out[pl.at(i) + c] + acc[i][j] : acc[i][j];
      }
  }
}

template <typename T, bool kVec, int kC>
__global__ void __launch_bounds__(max_threads(kC))
    norm_backward_kernel(const NormBackwardArgs a, int group) {
  pdl_wait();
  using P = Piece<T, kVec>;
  __shared__ Exchange ex;
  const Place pl(group);
  float acc[kC][8];
#pragma unroll
  for (int i = 0; i < kC; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
  int buf = 0;
  for (int64_t base = (int64_t)blockIdx.x * pl.per_block; base < a.rows; base += (int64_t)gridDim.x * pl.per_block, buf ^= 1) {
    const int64_t row = base + pl.sub;
    const bool live = row < a.rows;
    P dy[kC], h[kC], dh[kC];
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      const int n = live ? pl.cols(i, a.H) : 0;
      dy[i].load(static_cast<const T*>(a.d_y) + row * a.ld_d_y + pl.at(i), pl.l, n);
      h[i].load(static_cast<const T*>(a.h) + row * a.ld_h + pl.at(i), pl.l, n);
      if (a.d_h) dh[i].load(static_cast<const T*>(a.d_h) + row * a.ld_d_h + pl.at(i), pl.l, n);
    }
    const float rstd = live ? a.rstd[row] : 0.f;
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      float w[8];
      load_weights<T, kVec>(a.weight, a.w_fp32, pl.at(i), pl.l, pl.cols(i, a.H), w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float hj = h[i].at(j);
        dot = fmaf(dy[i].at(j) * w[j], hj, dot);
        acc[i][j] = fmaf(dy[i].at(j), hj * rstd, acc[i][j]);
      }
    }
    const float2 r = group_reduce<false>(dot, 0.f, group, ex, buf);
    const float c = rstd * rstd * (r.x / (float)a.H);  // mean(g h) rstd^2
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      float w[8], d[8];
      load_weights<T, kVec>(a.weight, a.w_fp32, pl.at(i), pl.l, pl.cols(i, a.H), w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        d[j] = rstd * fmaf(-h[i].at(j), c, dy[i].at(j) * w[j]);
        if (a.d_h) d[j] += dh[i].at(j);
      }
      P::store(static_cast<T*>(a.d_x) + row * a.H + pl.at(i), pl.l, live ? pl.cols(i, a.H) : 0, d);
    }
  }
  store_partial<kVec, kC>(a, pl, acc);
}

// The same with the rows in shared memory, which are read twice there; a stage is
// refilled after the next row's exchange, when every thread has left it.
template <typename T, int kC>
__global__ void __launch_bounds__(512, 1) norm_backward_ring_kernel(const NormBackwardArgs a, int group, const RingArgs r) {
  extern __shared__ __align__(128) uint8_t stage_smem[];
  using P = Piece<T, true>;
  __shared__ Ring ring;
  __shared__ Exchange ex;
  ring_init(ring, r);
  pdl_wait();
  const Place pl(group);
  const void* const mat[3] = {a.d_y, a.h, a.d_h};
  const int64_t size = sizeof(T), pitch[3] = {a.ld_d_y * size, a.ld_h * size, a.ld_d_h * size};
  const int64_t step = (int64_t)gridDim.x * pl.per_block, base0 = (int64_t)blockIdx.x * pl.per_block;
  if (threadIdx.x == 0)
    for (int s = 0; s < r.stages; ++s) ring_fill(ring, r, smem_u32(stage_smem), s, mat, pitch, base0 + s * step, a.rows, pl.per_block);
  float acc[kC][8];
  P w[kC];  // as loaded (all 1 without weights); FP32 weights of 16-bit rows stay in global memory
  const bool held = !a.w_fp32 || sizeof(T) == 4;
#pragma unroll
  for (int i = 0; i < kC; ++i) {
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
    if (a.weight && held) w[i].load(static_cast<const T*>(a.weight) + pl.at(i), pl.l, pl.cols(i, a.H));
  }
  auto weights = [&](int i, float (&f)[8]) {
    if (a.weight && held) {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = w[i].at(j);
    } else {
      load_weights<T, true>(a.weight, a.w_fp32, pl.at(i), pl.l, pl.cols(i, a.H), f);
    }
  };
  int stage = 0, buf = 0;
  uint32_t phase = 0;
  const float inv_H = 1.f / (float)a.H;
  for (int64_t base = base0; base < a.rows; base += step, buf ^= 1) {
    const int64_t row = base + pl.sub;
    const bool live = row < a.rows;
    const float rstd = live ? __ldg(a.rstd + row) : 0.f;
    mbar_wait(smem_u32(&ring.full[stage]), phase, r.ctl, &ring.abort);
    const T* sdy = reinterpret_cast<const T*>(stage_smem + stage * r.stage_bytes + pl.sub * r.row_bytes);
    const T* sh = reinterpret_cast<const T*>(reinterpret_cast<const uint8_t*>(sdy) + pl.per_block * r.row_bytes);
    const T* sdh = reinterpret_cast<const T*>(reinterpret_cast<const uint8_t*>(sh) + pl.per_block * r.row_bytes);
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      P dy, h;
      dy.load(sdy + pl.at(i), pl.l, live ? pl.cols(i, a.H) : 0);
      h.load(sh + pl.at(i), pl.l, live ? pl.cols(i, a.H) : 0);
      float f[8];
      weights(i, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float t = dy.at(j) * h.at(j);
        dot = fmaf(t, f[j], dot);
        acc[i][j] = fmaf(t, rstd, acc[i][j]);
      }
    }
    const float2 q = group_reduce<false>(dot, 0.f, group, ex, buf);
    if (pl.group <= 32) __syncthreads();
    if (threadIdx.x == 0 && base != base0) {  // every thread has left the stage of the row before
      const int64_t next = base + (r.stages - 1) * step;
      ring_fill(ring, r, smem_u32(stage_smem), stage ? stage - 1 : r.stages - 1, mat, pitch, next, a.rows, pl.per_block);
    }
    const float c = rstd * rstd * rstd * (q.x * inv_H);
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      const int n = live ? pl.cols(i, a.H) : 0;
      P dy, h, dh;
      dy.load(sdy + pl.at(i), pl.l, n);
      h.load(sh + pl.at(i), pl.l, n);
      if (a.d_h) dh.load(sdh + pl.at(i), pl.l, n);
      float f[8], d[8];
      weights(i, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        d[j] = fmaf(-h.at(j), c, dy.at(j) * (f[j] * rstd));
        if (a.d_h) d[j] += dh.at(j);
      }
      P::store(static_cast<T*>(a.d_x) + row * a.H + pl.at(i), pl.l, n, d);
    }
    if (++stage == r.stages) stage = 0, phase ^= 1;
  }
  store_partial<true, kC>(a, pl, acc);
}

// d_w[c] = sum of the `parts` partial sums of column c.  32 columns per block, 8
// lanes of partial sums each, which meet in a fixed order.
__global__ void __launch_bounds__(256) norm_weight_kernel(const float* __restrict__ partial, int parts, int64_t H,
                                                          float* __restrict__ d_w) {
  pdl_wait();
  __shared__ float s[8][32];
  const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x;
  float sum = 0.f;
  if (c < H) {
#pragma unroll 8
    for (int p = threadIdx.y; p < parts; p += 8) sum += partial[(int64_t)p * H + c];
  }
  s[threadIdx.y][threadIdx.x] = sum;
  __syncthreads();
  if (threadIdx.y == 0 && c < H) {
    for (int i = 1; i < 8; ++i) sum += s[i][threadIdx.x];
    d_w[c] = sum;
  }
}

// How rows are spread: kC pieces per thread, threads per row and per block, blocks,
// and the ring's stages (0: none) and bytes.
struct Shape {
  int C, group, threads, grid, stages;
  uint32_t stage_bytes;
};
Shape shape_of(int64_t rows, int64_t H, int mats, int size, bool vec) {
  const int blocks = (int)ceil_div(H, 128);
  auto spread = [&](int C, int most_threads) {
    Shape s = {};
    s.C = C;
    const int halves = (int)ceil_div(blocks, C);  // groups of 16 lanes
    s.group = halves == 1 ? 16 : (halves + 1) / 2 * 32;
    s.threads = std::max(1, most_threads / s.group) * s.group;
    return s;
  };
  const int64_t sms = num_sms();
  if (vec && blocks <= 128) {
    Shape s = spread(blocks >= 16 ? 4 : blocks >= 4 ? 2 : 1, 256);
    const int per_block = s.threads / s.group;
    s.stage_bytes = (uint32_t)(mats * per_block * H * size);
    const int resident = s.threads <= 256 && 2 * s.stage_bytes <= 108 * 1024 ? 2 : 1;
    s.stages = (int)std::min<int64_t>(kMaxRing, (resident == 2 ? 108 : 216) * 1024 / s.stage_bytes);
    s.grid = (int)std::min<int64_t>(ceil_div(rows, per_block), sms * resident);
    if (s.stages >= 2 && ceil_div(rows, per_block) >= 2 * sms * resident) return s;
  }
  int C = 1;
  const int most = rows <= 2 * sms ? 64 : 16;  // blocks of 128 columns that one piece per thread takes
  while (C < 8 && ceil_div(blocks, C) > (C == 1 ? most : 16)) C *= 2;
  Shape s = spread(C, 128);
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

// The kernel's shared memory is allowed once per device.
template <typename Kernel>
q4_status allow_smem(Kernel kernel, int (&ready)[64]) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return Q4_ERR_CUDA;
  if (!ready[dev]) {
    Q4_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 216 * 1024));
    ready[dev] = 1;
  }
  return Q4_OK;
}

RingArgs ring_of(const Shape& s, int64_t row_bytes) {
  return RingArgs{s.stages, s.stage_bytes, (uint32_t)row_bytes, KernelCtl{device_status_ptr(), wait_budget_ns()}};
}

template <typename T, int kC, int kForm>
q4_status launch_norm_ring(const NormArgs& a, const Shape& s, cudaStream_t stream) {
  static int ready[64] = {0};
  const q4_status st = allow_smem(norm_ring_kernel<T, kC, kForm>, ready);
  if (st != Q4_OK) return st;
  return launch_pdl(norm_ring_kernel<T, kC, kForm>, s.grid, s.threads, (size_t)s.stages * s.stage_bytes, stream, a, s.group,
                    ring_of(s, a.H * (int64_t)sizeof(T)));
}

template <typename T, int kC, int kForm>
q4_status launch_norm_form(const NormArgs& a, const Shape& s, bool vec, cudaStream_t stream) {
  if constexpr (kC <= 4)
    if (s.stages) return launch_norm_ring<T, kC, kForm>(a, s, stream);
  return launch_pdl(vec ? norm_kernel<T, true, kC, kForm> : norm_kernel<T, false, kC, kForm>, s.grid, s.threads, 0, stream, a,
                    s.group, device_status_ptr());
}

template <typename T, int kC>
q4_status launch_norm_backward_ring(const NormBackwardArgs& a, const Shape& s, cudaStream_t stream) {
  static int ready[64] = {0};
  const q4_status st = allow_smem(norm_backward_ring_kernel<T, kC>, ready);
  if (st != Q4_OK) return st;
  return launch_pdl(norm_backward_ring_kernel<T, kC>, s.grid, s.threads, (size_t)s.stages * s.stage_bytes, stream, a, s.group,
                    ring_of(s, a.H * (int64_t)sizeof(T)));
}

}  // namespace

q4_status launch_norm(const NormArgs& a, int dtype, int form, cudaStream_t stream) {
  const int size = dtype == Q4_F32 ? 4 : 2;
  const bool vec = a.H % 8 == 0 && a.ldx * size % 16 == 0 && (!a.residual || a.ld_residual * size % 16 == 0) && mult(a.x, 16) &&
                   mult(a.residual, 16) && mult(a.h, 16) && mult(a.y, 16) && mult(a.codes, 8) && mult(a.weight, 16);
  const Shape s = shape_of(a.rows, a.H, a.residual ? 2 : 1, size, vec);
  return by_dtype(dtype, [&](auto tag) {
    using T = decltype(tag);
    return by_pieces(s.C, [&](auto c) {
      constexpr int C = decltype(c)::value;
      if (form == Q4_NORM_FP8) return launch_norm_form<T, C, Q4_NORM_FP8>(a, s, vec, stream);
      if (form == Q4_NORM_INT8) return launch_norm_form<T, C, Q4_NORM_INT8>(a, s, vec, stream);
      return launch_norm_form<T, C, Q4_NORM_PLAIN>(a, s, vec, stream);
    });
  });
}

// Room for the largest grid that these sizes can have.
size_t norm_backward_workspace_bytes(int64_t rows, int64_t H) {
  if (rows == 0 || H == 0) return 0;
  int grid = 0;
  for (int mats : {2, 3})
    for (int size : {2, 4})
      for (bool vec : {false, true}) grid = std::max(grid, shape_of(rows, H, mats, size, vec).grid);
  return (size_t)grid * (size_t)H * sizeof(float);
}

q4_status launch_norm_backward(NormBackwardArgs a, int dtype, float* d_weight, void* ws, cudaStream_t stream) {
  a.partial = d_weight ? static_cast<float*>(ws) : nullptr;
  const int size = dtype == Q4_F32 ? 4 : 2;
  const bool vec = a.H % 8 == 0 && a.ld_d_y * size % 16 == 0 && a.ld_h * size % 16 == 0 && (!a.d_h || a.ld_d_h * size % 16 == 0) &&
                   mult(a.d_y, 16) && mult(a.h, 16) && mult(a.d_h, 16) && mult(a.d_x, 16) && mult(a.weight, 16);
  const Shape s = shape_of(a.rows, a.H, a.d_h ? 3 : 2, size, vec);
  const q4_status st = by_dtype(dtype, [&](auto tag) {
    using T = decltype(tag);
    return by_pieces(s.C, [&](auto c) {
      constexpr int C = decltype(c)::value;
      if constexpr (C <= 4)
        if (s.stages) return launch_norm_backward_ring<T, C>(a, s, stream);
      return launch_pdl(vec ? norm_backward_kernel<T, true, C> : norm_backward_kernel<T, false, C>, s.grid, s.threads, 0, stream, a,
                        s.group);
    });
  });
  if (st != Q4_OK || !d_weight) return st;
  return launch_pdl(norm_weight_kernel, (unsigned)ceil_div(a.H, 32), dim3(32, 8), 0, stream, static_cast<const float*>(ws), s.grid,
                    a.H, d_weight);
}

}  // namespace q4
