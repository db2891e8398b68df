// Gradient of the root-mean-square norm.  With g = d_y w,
//   d_x = rstd g - h rstd^3 mean(g h) (+ d_h),  d_w = sum over rows of d_y h rstd
//
// Each block of threads takes every gridDim.x-th row (or as many rows as it has
// groups) and adds its rows' part of d_w up in registers, columns fixed to
// threads; the blocks' sums go to the workspace and are added in their order by
// a second kernel, so that results do not depend on timing.
//
// HBM-bound where rows are aligned: 16384 x 7168 bf16 with d_h 150.9 us (6.2 TB/s; with
// FP32 weights, read for every row, 182), 8192 x 4096 50.6 us (5.3 TB/s); single elements
// wait for their latencies: 9973 x 1411 bf16 36.2 us (2.3 TB/s), FP32 36.6 (4.6 TB/s).
// 512 x 4096 11.8 us, 64 x 16384 16.2: latencies of two dependent kernels; 65536 x 128
// without d_h 18.6 (2.7 TB/s): the same of short rows.
#include "rows.cuh"

namespace q4 {
namespace {

// rstd^3 mean, by factors that stay in range: rstd mean is as large as g (rstd^3 by
// itself is below the least number for h above 2^49).
__device__ __forceinline__ float h_factor(float rstd, float mean) { return rstd * (rstd * (rstd * mean)); }

// The block's part of d_w: the groups' sums, added up in their order by the first
// (one after another in global memory 65536 x 128 25.3 us instead of 18.4).
// scratch: 8 words per thread of shared memory that nothing else uses any more.
template <bool kVec, int kC>
__device__ __forceinline__ void store_partial(const NormBackwardArgs& a, const Place& pl, float (&acc)[kC][8], float* scratch) {
  if (!a.partial) return;
  if (pl.per_block > 1) {
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      __syncthreads();  // every thread has left the memory
      if (pl.sub) {
#pragma unroll
        for (int j = 0; j < 8; ++j) scratch[j * blockDim.x + threadIdx.x] = acc[i][j];
      }
      __syncthreads();
      if (pl.sub) continue;
      for (int s = 1; s < pl.per_block; ++s)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] += scratch[j * blockDim.x + s * pl.group + pl.t];
    }
    if (pl.sub) return;
  }
  float* out = a.partial + (int64_t)blockIdx.x * a.H;
#pragma unroll
  for (int i = 0; i < kC; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = kVec ? 8 * pl.l + j : pl.l + 16 * j;
      if (c < pl.cols(i, (int)a.H)) out[pl.at(i) + c] = acc[i][j];
    }
}

template <typename T, bool kVec, int kC>
__global__ void __launch_bounds__(max_threads(kC))
    norm_backward_kernel(const NormBackwardArgs a, int group) {
  pdl_wait();
  using P = Piece<T, kVec>;
  // A row stays in registers between the two passes where there is room beside d_w's
  // sums, else it is read again, from L2 (2048 x 32768 bf16 206 us, held 592; 1000 x 7001 49
  // and 58).
  constexpr bool kHold = kC * P::words <= 16;
  __shared__ Exchange ex;
  exchange_init(ex);
  __syncthreads();
  const Place pl(group);
  const int width = (int)a.H;
  const float inv_H = 1.f / (float)width;
  float acc[kC][8];
#pragma unroll
  for (int i = 0; i < kC; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
  int buf = 0;
  for (int64_t base = (int64_t)blockIdx.x * pl.per_block; base < a.rows; base += (int64_t)gridDim.x * pl.per_block, buf ^= 1) {
    const int64_t row = base + pl.sub;
    const int H = row < a.rows ? width : 0;
    constexpr int kHeld = kHold ? kC : 1;
    P dy[kHeld], h[kHeld], dh[kHeld];
    auto load = [&](int i, bool join) {
      const int n = pl.cols(i, H), at = kHold ? i : 0;
      dy[at].load(static_cast<const T*>(a.d_y) + row * a.ld_d_y + pl.at(i), pl.l, n);
      h[at].load(static_cast<const T*>(a.h) + row * a.ld_h + pl.at(i), pl.l, n);
      if (join) dh[at].load(static_cast<const T*>(a.d_h) + row * a.ld_d_h + pl.at(i), pl.l, n);
    };
    if constexpr (kHold) {
#pragma unroll
      for (int i = 0; i < kC; ++i) load(i, a.d_h != nullptr);
    }
    const float rstd = H ? a.rstd[row] : 0.f;
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      if (!kHold) load(i, false);
      const int at = kHold ? i : 0;
      float w[8];
      load_weights<T, kVec>(a.weight, a.w_dtype == Q4_F32, pl.at(i), pl.l, pl.cols(i, width), w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float t = dy[at].at(j) * h[at].at(j);
        dot = fmaf(t, w[j], dot);
        acc[i][j] = fmaf(t, rstd, acc[i][j]);
      }
    }
    const float2 r = group_reduce<false>(dot, 0.f, group, ex, buf);
    const float c = h_factor(rstd, r.x * inv_H);
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      if (!kHold) load(i, a.d_h != nullptr);
      const int at = kHold ? i : 0;
      float w[8], d[8];
      load_weights<T, kVec>(a.weight, a.w_dtype == Q4_F32, pl.at(i), pl.l, pl.cols(i, width), w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        d[j] = fmaf(-h[at].at(j), c, dy[at].at(j) * (w[j] * rstd));
        if (a.d_h) d[j] += dh[at].at(j);
      }
      P::store(static_cast<T*>(a.d_x) + row * a.H + pl.at(i), pl.l, pl.cols(i, H), d);
    }
  }
  __shared__ float scratch[8 * max_threads(kC)];
  store_partial<kVec, kC>(a, pl, acc, scratch);
}

// The same with the rows in shared memory, which aligned ones are read from twice;
// a stage is refilled after the next row's exchange, when every thread has left it.
template <typename T, bool kVec, int kC, int kThreads>
__global__ void __launch_bounds__(kThreads, resident_blocks(kVec, kThreads, true))
    norm_backward_ring_kernel(const NormBackwardArgs a, int group, const RingArgs r) {
  extern __shared__ __align__(128) uint8_t stage_smem[];
  using P = Piece<T, kVec>;
  // between the two passes in registers (aligned rows, of 32 elements per thread, have
  // none for it: 16384 x 7168 bf16 154 us without and 201 with, then)
  constexpr bool kHold = !kVec;
  __shared__ Ring ring;
  __shared__ Exchange ex;
  ring_init(ring, r, ex);
  pdl_wait();
  const Place pl(group);
  const int width = (int)a.H;
  const float inv_H = 1.f / (float)width;
  const void* const mat[3] = {a.d_y, a.h, a.d_h};
  const int64_t size = sizeof(T), pitch[3] = {a.ld_d_y * size, a.ld_h * size, a.ld_d_h * size};
  const int64_t step = (int64_t)gridDim.x * pl.per_block, base0 = (int64_t)blockIdx.x * pl.per_block;
  if (threadIdx.x == 0)
    for (int s = 0; s < r.stages; ++s)
      ring_fill<kVec>(ring, r, smem_u32(stage_smem), s, mat, pitch, base0 + s * step, a.rows, pl.per_block);
  const HeldWeights<T, kVec, kC> w(a.weight, a.w_dtype, pl, width);
  float acc[kC][8];
#pragma unroll
  for (int i = 0; i < kC; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
  int stage = 0, buf = 0;
  uint32_t phase = 0;
  auto rows = [&](auto tag) {
    constexpr bool kWhole = decltype(tag)::value;  // as in the forward kernel
    for (int64_t base = base0; base < a.rows; base += step, buf ^= 1) {
      const int64_t row = base + pl.sub;
      const int H = kWhole || row < a.rows ? width : 0;
      const float rstd = kWhole || H ? __ldg(a.rstd + row) : 0.f;
      mbar_wait(smem_u32(&ring.full[stage]), phase, r.ctl, &ring.abort);
      const uint8_t* st = stage_smem + stage * r.stage_bytes;
      const T* dy_row = ring_row<kVec, T>(st, r, 0, pl, a.d_y, pitch[0], row);
      const T* h_row = ring_row<kVec, T>(st, r, 1, pl, a.h, pitch[1], row);
      const T* dh_row = ring_row<kVec, T>(st, r, 2, pl, a.d_h, pitch[2], row);
      if (!kVec && read_in_place(row, a.rows, r.edge)) {
        dy_row = static_cast<const T*>(a.d_y) + row * a.ld_d_y;
        h_row = static_cast<const T*>(a.h) + row * a.ld_h;
        dh_row = static_cast<const T*>(a.d_h) + row * a.ld_d_h;
      }
      float dot = 0.f;
      P held_dy[kHold ? kC : 1], held_h[kHold ? kC : 1];
#pragma unroll
      for (int i = 0; i < kC; ++i) {
        const int n = kWhole ? 128 : pl.cols(i, H);
        P& dy = held_dy[kHold ? i : 0];
        P& h = held_h[kHold ? i : 0];
        float f[8];
        dy.load(dy_row + pl.at(i), pl.l, n);
        h.load(h_row + pl.at(i), pl.l, n);
        w.template get<kWhole>(pl, width, i, f);
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
        const int left = stage ? stage - 1 : r.stages - 1;
        if (ring_over(ring, left, stage ? phase : phase ^ 1))
          ring_fill<kVec>(ring, r, smem_u32(stage_smem), left, mat, pitch, next, a.rows, pl.per_block);
      }
      const float c = h_factor(rstd, q.x * inv_H);
      T* out = static_cast<T*>(a.d_x) + row * a.H;
#pragma unroll
      for (int i = 0; i < kC; ++i) {
        const int n = kWhole ? 128 : pl.cols(i, H);
        P& dy = held_dy[kHold ? i : 0];
        P& h = held_h[kHold ? i : 0];
        float f[8];
        if (!kHold) {
          dy.load(dy_row + pl.at(i), pl.l, n);
          h.load(h_row + pl.at(i), pl.l, n);
        }
        w.template get<kWhole>(pl, width, i, f);
        float d[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = fmaf(-h.at(j), c, dy.at(j) * (f[j] * rstd));
        if (a.d_h) {
          P dh;
          dh.load(dh_row + pl.at(i), pl.l, n);
#pragma unroll
          for (int j = 0; j < 8; ++j) d[j] += dh.at(j);
        }
        P::store(out + pl.at(i), pl.l, n, d);
      }
      if (++stage == r.stages) stage = 0, phase ^= 1;
    }
  };
  if constexpr (kVec && kC == 4) {
    if (w.held && pl.whole(kC, width) && a.rows % pl.per_block == 0)
      rows(std::true_type());
    else
      rows(std::false_type());
  } else {
    rows(std::false_type());
  }
  ring_end(ring, r);
  store_partial<kVec, kC>(a, pl, acc, reinterpret_cast<float*>(stage_smem));
}

// d_w[c] = sum of the `parts` partial sums of column c.  32 columns per block, 32
// warps of partial sums each, which meet in a fixed order (8 warps: 10 us instead
// of 3 for 304 parts of 7168).
constexpr int kWeightWarps = 32;
__global__ void __launch_bounds__(32 * kWeightWarps) norm_weight_kernel(const float* __restrict__ partial, int parts, int64_t H,
                                                                        float* __restrict__ d_w) {
  pdl_wait();
  __shared__ float s[kWeightWarps][33];
  const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x;
  float sum = 0.f;
  if (c < H) {
#pragma unroll 8
    for (int p = threadIdx.y; p < parts; p += kWeightWarps) sum += partial[(int64_t)p * H + c];
  }
  s[threadIdx.y][threadIdx.x] = sum;
  __syncthreads();
  // warp y adds the parts of column y up
  sum = s[threadIdx.x][threadIdx.y];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const int64_t mine = (int64_t)blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && mine < H) d_w[mine] = sum;
}

template <typename T, bool kVec, int kC, int kThreads>
q4_status launch_norm_backward_ring(const NormBackwardArgs& a, const Shape& s, cudaStream_t stream) {
  static std::atomic<int> ready[64];
  const auto kernel = norm_backward_ring_kernel<T, kVec, kC, kThreads>;
  const q4_status st = allow_smem(kernel, ready);
  if (st != Q4_OK) return st;
  const uint32_t scratch = s.threads > s.group ? 32 * (uint32_t)s.threads : 0;
  return launch_pdl(kernel, s.grid, s.threads, std::max(s.stages * s.stage_bytes, scratch), stream, a, s.group,
                    ring_of(s, kVec, a.H * (int64_t)sizeof(T)));
}

template <typename T, int kC>
q4_status launch_norm_backward_form(const NormBackwardArgs& a, const Shape& s, bool vec, cudaStream_t stream) {
  if (s.stages) {
    if constexpr (kC == 2)
      if (!vec) return launch_norm_backward_ring<T, false, kC, 256>(a, s, stream);
    if constexpr (kC == 4)
      if (s.threads > 256) return launch_norm_backward_ring<T, true, kC, 512>(a, s, stream);
    if constexpr (kC <= 4) return launch_norm_backward_ring<T, true, kC, 256>(a, s, stream);
  }
  if constexpr (kC != 2)
    return launch_pdl(vec ? norm_backward_kernel<T, true, kC> : norm_backward_kernel<T, false, kC>, s.grid, s.threads, 0, stream, a,
                      s.group);
  return Q4_ERR_UNSUPPORTED_SHAPE;  // not reached: two pieces are for rings
}

}  // namespace

namespace {
// The gradient's spread: where rows are few, at most a block per SM, since each
// writes a row of d_w's parts (512 x 4096: 19 us with a block per row), and as many
// rows at a time in it (11.7 us, one after another 17.0).
Shape backward_shape(int64_t rows, int64_t H, int mats, int size, bool vec) {
  Shape s = shape_of(rows, H, mats, size, vec, true);
  if (s.stages) return s;
  const int64_t most = std::min(max_threads(s.C) / s.group, most_groups(s.group));
  const int64_t side = std::min<int64_t>(ceil_div(rows, num_sms()), most);
  s.threads = (int)std::max<int64_t>(side, 1) * s.group;
  s.grid = (int)std::min<int64_t>(ceil_div(rows, s.threads / s.group), num_sms());
  return s;
}
}  // namespace

// Room for the largest grid: at most two blocks per SM, a row or more each.
size_t norm_backward_workspace_bytes(int64_t rows, int64_t H) {
  if (rows == 0 || H == 0) return 0;
  return (size_t)std::min<int64_t>(rows, 2 * num_sms()) * (size_t)H * sizeof(float);
}

q4_status launch_norm_backward(NormBackwardArgs a, int dtype, float* d_weight, void* ws, cudaStream_t stream) {
  a.partial = d_weight ? static_cast<float*>(ws) : nullptr;
  const int size = dtype == Q4_F32 ? 4 : 2;
  const bool vec = a.H % 8 == 0 && a.ld_d_y * size % 16 == 0 && a.ld_h * size % 16 == 0 && (!a.d_h || a.ld_d_h * size % 16 == 0) &&
                   mult(a.d_y, 16) && mult(a.h, 16) && mult(a.d_h, 16) && mult(a.d_x, 16) && mult(a.weight, 16);
  const Shape s = backward_shape(a.rows, a.H, a.d_h ? 3 : 2, size, vec);
  const q4_status st = by_dtype(dtype, [&](auto tag) {
    using T = decltype(tag);
    return by_pieces(s.C, [&](auto c) {
      return launch_norm_backward_form<T, decltype(c)::value>(a, s, vec, stream);
    });
  });
  if (st != Q4_OK || !d_weight) return st;
  return launch_pdl(norm_weight_kernel, (unsigned)ceil_div(a.H, 32), dim3(32, kWeightWarps), 0, stream, static_cast<const float*>(ws), s.grid,
                    a.H, d_weight);
}

}  // namespace q4
