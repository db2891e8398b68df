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
// pieces each.
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
// Groups of more than a warp are the whole block; buf alternates between two
// buffers from row to row, so that one barrier per row is enough.
struct Exchange {
  float2 part[2][32];
};
__device__ __forceinline__ float2 group_reduce(float sum, float top, int group, Exchange& ex, int buf) {
  const int width = min(group, 32);
  for (int o = width / 2; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  }
  if (group > 32) {
    const int lane = threadIdx.x & 31, warps = group >> 5;
    if (lane == 0) ex.part[buf][threadIdx.x >> 5] = make_float2(sum, top);
    __syncthreads();
    const float2 v = lane < warps ? ex.part[buf][lane] : make_float2(0.f, 0.f);
    sum = v.x, top = v.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      sum += __shfl_xor_sync(0xffffffffu, sum, o);
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
  }
  return make_float2(sum, top);
}

// Threads of a block for kC pieces per thread.
constexpr int max_threads(int C) { return C == 1 ? 1024 : 512; }

template <typename T, bool kVec, int kC, int kForm>
__global__ void __launch_bounds__(max_threads(kC))
    norm_kernel(const NormArgs a, int group, int* status) {
  pdl_wait();
  using P = Piece<T, kVec>;
  __shared__ Exchange ex;
  const int l = threadIdx.x & 15, t = threadIdx.x & (group > 32 ? ~0 : group - 1);
  const int per_block = blockDim.x / group;  // rows
  const int sub = group > 32 ? 0 : threadIdx.x / group;
  const int blocks = (int)((a.H + 127) / 128), stride = group >> 4;
  const T* x = static_cast<const T*>(a.x);
  const T* res = static_cast<const T*>(a.residual);
  constexpr bool kKeep = kC <= 4;  // the weights stay in registers from row to row
  float w[kKeep ? kC : 1][8];
  auto weights = [&](int i, float (&f)[8]) {
    const int b = (t >> 4) + i * stride;
    load_weights<T, kVec>(a.weight, a.w_fp32, (int64_t)b * 128, l, (int)min((int64_t)128, a.H - (int64_t)b * 128), f);
  };
  if constexpr (kKeep) {
#pragma unroll
    for (int i = 0; i < kC; ++i) weights(i, w[i]);
  }
  int buf = 0;
  for (int64_t base = (int64_t)blockIdx.x * per_block; base < a.rows; base += (int64_t)gridDim.x * per_block, buf ^= 1) {
    const int64_t row = base + sub;
    const bool live = row < a.rows;
    // columns of piece i; none behind the row's last block or the last row
    auto cols = [&](int i) {
      const int b = (t >> 4) + i * stride;
      return live ? (int)min((int64_t)128, a.H - (int64_t)b * 128) : 0;
    };
    auto at = [&](int i) { return (int64_t)((t >> 4) + i * stride) * 128; };
    float v[kC][8];  // h, then h w
    float sum = 0.f, top = 0.f;
    {
      P px[kC], pr[kC];
#pragma unroll
      for (int i = 0; i < kC; ++i) px[i].load(x + row * a.ldx + at(i), l, cols(i));
      if (res) {
#pragma unroll
        for (int i = 0; i < kC; ++i) pr[i].load(res + row * a.ld_residual + at(i), l, cols(i));
      }
#pragma unroll
      for (int i = 0; i < kC; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = res ? px[i].at(j) + pr[i].at(j) : px[i].at(j);
    }
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      if (a.h) P::store(static_cast<T*>(a.h) + row * a.H + at(i), l, cols(i), v[i]);
      float wi[8];
      if constexpr (!kKeep) weights(i, wi);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        sum = fmaf(v[i][j], v[i][j], sum);
        v[i][j] *= kKeep ? w[kKeep ? i : 0][j] : wi[j];
        if (kForm == Q4_NORM_INT8) top = fmaxf(top, fabsf(v[i][j]));
      }
    }
    const float2 r = group_reduce(sum, top, group, ex, buf);
    const float rstd = __frsqrt_rn(r.x / (float)a.H + a.eps);
    if (t == 0 && live) {
      if (a.rstd) a.rstd[row] = rstd;
      if (nonfinite(r.x)) latch_status(status, Q4_ERR_NONFINITE);
    }
    if constexpr (kForm == Q4_NORM_INT8) {
      const float s = __fdiv_rn(fmaxf(r.y * rstd, 1e-12f), 127.f);
      if (t == 0 && live) {
        a.scales[row] = s;
        if (nonfinite(s)) latch_status(status, Q4_ERR_NONFINITE);
      }
      const float f = __fdiv_rn(rstd, s);
#pragma unroll
      for (int i = 0; i < kC; ++i) P::store_codes(a.codes + row * a.H + at(i), l, cols(i), int8x8(v[i], f));
    }
    if constexpr (kForm == Q4_NORM_FP8) {
#pragma unroll
      for (int i = 0; i < kC; ++i) {
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[i][j]));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float s = __fdiv_rn(fmaxf(m * rstd, 1e-12f), 448.f);
        P::store_codes(a.codes + row * a.H + at(i), l, cols(i), e4m3x8(v[i], __fdiv_rn(rstd, s)));
        if (l == 0 && cols(i) > 0) {
          a.scales[row * blocks + (t >> 4) + i * stride] = s;
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
        P::store(static_cast<T*>(a.y) + row * a.H + at(i), l, cols(i), y);
      }
    }
  }
}

// ------------------------------------------------------------------ gradient
// Each block of threads takes every gridDim.x-th row (or as many rows as it has
// groups) and adds its rows' part of d_w up in registers, columns fixed to
// threads; the blocks' sums go to the workspace and are added in their order by
// a second kernel, so that results do not depend on timing.
template <typename T, bool kVec, int kC>
__global__ void __launch_bounds__(max_threads(kC))
    norm_backward_kernel(const NormBackwardArgs a, int group) {
  pdl_wait();
  using P = Piece<T, kVec>;
  __shared__ Exchange ex;
  const int l = threadIdx.x & 15, t = threadIdx.x & (group > 32 ? ~0 : group - 1);
  const int per_block = blockDim.x / group;
  const int sub = group > 32 ? 0 : threadIdx.x / group;
  const int stride = group >> 4;
  auto at = [&](int i) { return (int64_t)((t >> 4) + i * stride) * 128; };
  auto width = [&](int i) { return (int)min((int64_t)128, a.H - at(i)); };
  float acc[kC][8];
#pragma unroll
  for (int i = 0; i < kC; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
  int buf = 0;
  for (int64_t base = (int64_t)blockIdx.x * per_block; base < a.rows; base += (int64_t)gridDim.x * per_block, buf ^= 1) {
    const int64_t row = base + sub;
    const bool live = row < a.rows;
    P dy[kC], h[kC], dh[kC];
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      const int n = live ? width(i) : 0;
      dy[i].load(static_cast<const T*>(a.d_y) + row * a.ld_d_y + at(i), l, n);
      h[i].load(static_cast<const T*>(a.h) + row * a.ld_h + at(i), l, n);
      if (a.d_h) dh[i].load(static_cast<const T*>(a.d_h) + row * a.ld_d_h + at(i), l, n);
    }
    const float rstd = live ? a.rstd[row] : 0.f;
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      float w[8];
      load_weights<T, kVec>(a.weight, a.w_fp32, at(i), l, width(i), w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float hj = h[i].at(j);
        dot = fmaf(dy[i].at(j) * w[j], hj, dot);
        acc[i][j] = fmaf(dy[i].at(j), hj * rstd, acc[i][j]);
      }
    }
    const float2 r = group_reduce(dot, 0.f, group, ex, buf);
    const float c = rstd * rstd * (r.x / (float)a.H);  // mean(g h) rstd^2
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      float w[8], d[8];
      load_weights<T, kVec>(a.weight, a.w_fp32, at(i), l, width(i), w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        d[j] = rstd * fmaf(-h[i].at(j), c, dy[i].at(j) * w[j]);
        if (a.d_h) d[j] += dh[i].at(j);
      }
      P::store(static_cast<T*>(a.d_x) + row * a.H + at(i), l, live ? width(i) : 0, d);
    }
  }
  if (!a.partial) return;
  // the block's groups one after another: group s writes (s = 0) or adds
  float* out = a.partial + (int64_t)blockIdx.x * a.H;
  for (int s = 0; s < per_block; ++s) {
    if (s) __syncthreads();
    if (sub != s) continue;
#pragma unroll
    for (int i = 0; i < kC; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int c = kVec ? 8 * l + j : l + 16 * j;
        if (c < width(i)) out[at(i) + c] = s ? out[at(i) + c] + acc[i][j] : acc[i][j];
      }
  }
}

// d_w[c] = sum of the `parts` partial sums of column c.  32 columns per block, 8
// lanes of partial sums each, which meet in a fixed order.
__global__ void __launch_bounds__(256) norm_weight_kernel(const float* __restrict__ partial, int parts, int64_t H,
                                                          float* __restrict__ d_w) {
  pdl_wait();
  __shared__ float s[8][32];
  const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x;
  float sum = 0.f;
  if (c < H)
    for (int p = threadIdx.y; p < parts; p += 8) sum += partial[(int64_t)p * H + c];
  s[threadIdx.y][threadIdx.x] = sum;
  __syncthreads();
  if (threadIdx.y == 0 && c < H) {
    for (int i = 1; i < 8; ++i) sum += s[i][threadIdx.x];
    d_w[c] = sum;
  }
}

// How a row is spread: kC pieces per thread, threads per row, threads per block.
struct Shape {
  int C, group, threads;
};
Shape shape_of(int64_t rows, int64_t H) {
  const int blocks = (int)ceil_div(H, 128);
  Shape s;
  s.C = 1;
  const int most = rows <= 2 * num_sms() ? 64 : 16;  // blocks of 128 columns that one piece per thread takes
  while (s.C < 8 && ceil_div(blocks, s.C) > (s.C == 1 ? most : 16)) s.C *= 2;
  const int halves = (int)ceil_div(blocks, s.C);  // groups of 16 lanes
  s.group = halves == 1 ? 16 : (halves + 1) / 2 * 32;
  s.threads = s.group > 32 ? s.group : 128;
  return s;
}

template <typename F>
q4_status by_pieces(int C, F&& f) {
  if (C == 1) return f(std::integral_constant<int, 1>());
  if (C == 2) return f(std::integral_constant<int, 2>());
  if (C == 4) return f(std::integral_constant<int, 4>());
  return f(std::integral_constant<int, 8>());
}

// Blocks of threads: as many as are resident, each going on to further rows.
int grid_of(const Shape& s, int64_t rows) {
  const int64_t need = ceil_div(rows, s.threads / s.group);
  return (int)std::min<int64_t>(need, (int64_t)num_sms() * std::max(1, 1024 / s.threads));
}

}  // namespace

q4_status launch_norm(const NormArgs& a, int dtype, int form, cudaStream_t stream) {
  const Shape s = shape_of(a.rows, a.H);
  const int64_t size = dtype == Q4_F32 ? 4 : 2;
  const bool vec = a.H % 8 == 0 && a.ldx * size % 16 == 0 && (!a.residual || a.ld_residual * size % 16 == 0) && mult(a.x, 16) &&
                   mult(a.residual, 16) && mult(a.h, 16) && mult(a.y, 16) && mult(a.codes, 8) && mult(a.weight, 16);
  return by_dtype(dtype, [&](auto tag) {
    using T = decltype(tag);
    return by_pieces(s.C, [&](auto c) {
      constexpr int C = decltype(c)::value;
      auto launch = [&](auto kernel) {
        return launch_pdl(kernel, grid_of(s, a.rows), s.threads, 0, stream, a, s.group, device_status_ptr());
      };
      if (form == Q4_NORM_FP8) return vec ? launch(norm_kernel<T, true, C, Q4_NORM_FP8>) : launch(norm_kernel<T, false, C, Q4_NORM_FP8>);
      if (form == Q4_NORM_INT8) return vec ? launch(norm_kernel<T, true, C, Q4_NORM_INT8>) : launch(norm_kernel<T, false, C, Q4_NORM_INT8>);
      return vec ? launch(norm_kernel<T, true, C, Q4_NORM_PLAIN>) : launch(norm_kernel<T, false, C, Q4_NORM_PLAIN>);
    });
  });
}

size_t norm_backward_workspace_bytes(int64_t rows, int64_t H) {
  if (rows == 0 || H == 0) return 0;
  return (size_t)grid_of(shape_of(rows, H), rows) * (size_t)H * sizeof(float);
}

q4_status launch_norm_backward(NormBackwardArgs a, int dtype, float* d_weight, void* ws, cudaStream_t stream) {
  const Shape s = shape_of(a.rows, a.H);
  const int grid = grid_of(s, a.rows);
  a.partial = d_weight ? static_cast<float*>(ws) : nullptr;
  const int64_t size = dtype == Q4_F32 ? 4 : 2;
  const bool vec = a.H % 8 == 0 && a.ld_d_y * size % 16 == 0 && a.ld_h * size % 16 == 0 && (!a.d_h || a.ld_d_h * size % 16 == 0) &&
                   mult(a.d_y, 16) && mult(a.h, 16) && mult(a.d_h, 16) && mult(a.d_x, 16) && mult(a.weight, 16);
  const q4_status st = by_dtype(dtype, [&](auto tag) {
    using T = decltype(tag);
    return by_pieces(s.C, [&](auto c) {
      constexpr int C = decltype(c)::value;
      return launch_pdl(vec ? norm_backward_kernel<T, true, C> : norm_backward_kernel<T, false, C>, grid, s.threads, 0, stream,
                        a, s.group);
    });
  });
  if (st != Q4_OK || !d_weight) return st;
  return launch_pdl(norm_weight_kernel, (unsigned)ceil_div(a.H, 32), dim3(32, 8), 0, stream, static_cast<const float*>(ws), grid,
                    a.H, d_weight);
}

}  // namespace q4
