// Activations kept in 8 bits for the backward pass, and the gated activation
// that writes and reads them.
//
// A checkpoint of x [rows, K] is E4M3 codes with one FP32 scale per row and
// 128 columns (the last block of a row may be shorter).  The scale is a power
// of two, the smallest s = 2^e with max(amax, 1e-12) <= 448 s: a code has four
// significant bits, so code * s is a bf16 number and the backward pass can
// feed it to the bf16 tensor cores without a second rounding, while against
// s = amax / 448 at most one bit of E4M3's range (none of its precision) is
// given up.  x / s is exact, so the only rounding is the E4M3 one (to nearest
// even; finite numbers of 248 * 2^120 and more stop at 240 * 2^120).
//
// swiglu of gate_up = [g | u]:  h = silu(g) u,  silu(g) = g / (1 + exp(-g));
// its gradient at the restored g and u, with s = 1 / (1 + exp(-g)):
//   dg = dh u s (1 + g (1 - s)),  du = dh g s.
#include <algorithm>

#include "common.cuh"
#include "elem.cuh"
#include "internal.h"

namespace q4 {
namespace {

constexpr int kThreads = 256;

// The values of the two codes in the low 16 bits.
__device__ __forceinline__ float2 e4m3x2_values(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// The largest scale's exponent.  Numbers from 248 * 2^120 on round to the code 256,
// which would stand for 2^128, beyond FP32 and bf16; they stop at 240.  (Greater
// codes come from infinities only, and stay.)
constexpr int kTopExponent = 120;

// Exponent of the block's scale: 448 = 1.75 * 2^8, so the significand of amax
// decides between its own exponent - 8 and - 7.
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t b = max(__float_as_uint(amax), __float_as_uint(1e-12f));
  return min((int)((b + 0x1fffffu) >> 23) - 127 - 8, kTopExponent);  // a non-finite block has the top one, too
}
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// silu's factor 1 / (1 + exp(-g)) with the fast exponential and reciprocal
// (below 2^-17 relative error for |g| <= 88; below g = -87.3 it is 0 instead
// of less than 1e-37).  The exact functions cost more issue slots than the
// whole rest of the kernels.
__device__ __forceinline__ float sigmoid(float g) { return __fdividef(1.f, 1.f + __expf(-g)); }

// A block of 128 columns is held by `lanes` lanes, `n` columns each.  With
// 128-bit accesses (kVec) a lane holds chunks of 8 columns, lanes * 8 apart: one
// chunk of FP32 (16 lanes), two of 16-bit elements (8 lanes), so that two loads
// are in flight either way (one chunk of bf16: swiglu_fp8 94 us instead of 79
// at 32768 x 2 x 2048).  Otherwise lane l of kSingle holds columns l, l +
// kSingle, ... one by one, 16-bit elements by way of whole registers (loads into
// half a register wait for one another); sixteen lanes suit the kernels that
// reduce over the block (quantize_fp8_checkpoint of 9973 x 2822 bf16: 23 us
// instead of 32 with a warp), a warp the gradient (27 us instead of 30 at 9973 x
// 1411; with a path without tests for whole blocks 30).  Columns past the
// block's end are zero; 16-bit elements of chunks stay packed in the words they
// were loaded as until they are used.
template <typename T, bool kVec, int kSingle>
struct Held {
  static constexpr int lanes = !kVec ? kSingle : sizeof(T) == 2 ? 8 : 16, n = 128 / lanes;
  static constexpr int chunks = kVec ? n / 8 : 1;
  static_assert(chunks * lanes * 8 == 128 || !kVec, "a block");
  static constexpr bool packed = kVec && sizeof(T) == 2;
  static constexpr int words = packed ? n / 2 : n;
  uint32_t w[words];

  static __device__ __forceinline__ int chunk(int l, int c) { return 8 * (l + lanes * c); }

  __device__ __forceinline__ void load(const T* __restrict__ p, int l, int cols) {
    if constexpr (kVec) {
      constexpr int per = words / chunks / 4;  // 128-bit words of a chunk
#pragma unroll
      for (int i = 0; i < words / 4; ++i) {
        const int at = chunk(l, i / per);
        const uint4 v = at < cols ? __ldg(reinterpret_cast<const uint4*>(p + at) + i % per) : make_uint4(0u, 0u, 0u, 0u);
        w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const int at = l + lanes * i;
        if constexpr (sizeof(T) == 2)
          w[i] = at < cols ? __ldg(reinterpret_cast<const unsigned short*>(p) + at) : 0u;
        else
          w[i] = at < cols ? __float_as_uint(__ldg(p + at)) : 0u;
      }
    }
  }
  __device__ __forceinline__ void floats(float (&f)[n]) const {
    if constexpr (packed) {
#pragma unroll
      for (int i = 0; i < words; ++i) {
        const float2 v = unpack2<T>(w[i]);
        f[2 * i] = v.x, f[2 * i + 1] = v.y;
      }
    } else if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < n; ++i) f[i] = unpack2<T>(w[i]).x;
    } else {
#pragma unroll
      for (int i = 0; i < n; ++i) f[i] = __uint_as_float(w[i]);
    }
  }
  // The block's largest magnitude, in every lane.  Taken on the bit patterns
  // without their sign, where infinities and NaN come out on top.
  __device__ __forceinline__ float amax() const {
    uint32_t top = 0;
    if constexpr (packed) {
#pragma unroll
      for (int i = 0; i < words; ++i) top = __vmaxu2(top, w[i] & 0x7fff7fffu);
#pragma unroll
      for (int o = lanes / 2; o > 0; o >>= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float2 v = unpack2<T>(top);  // NaN compares false, so it is kept if either half has it
      return __float_as_uint(v.x) > __float_as_uint(v.y) ? v.x : v.y;
    } else {
      constexpr uint32_t kMagnitude = sizeof(T) == 2 ? 0x7fffu : 0x7fffffffu;
#pragma unroll
      for (int i = 0; i < words; ++i) top = max(top, w[i] & kMagnitude);
#pragma unroll
      for (int o = lanes / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      if constexpr (sizeof(T) == 2)
        return unpack2<T>(top).x;
      else
        return __uint_as_float(top);
    }
  }

  static __device__ __forceinline__ void store(T* __restrict__ p, int l, int cols, const float (&v)[n]) {
    if constexpr (kVec) {
#pragma unroll
      for (int c = 0; c < chunks; ++c) {
        const int at = chunk(l, c);
        if (at >= cols) continue;
        uint4* out = reinterpret_cast<uint4*>(p + at);
        const float* f = v + 8 * c;
        if constexpr (sizeof(T) == 4) {
          out[0] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
          out[1] = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
        } else {
          out[0] = make_uint4(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]), pack2<T>(f[4], f[5]), pack2<T>(f[6], f[7]));
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < n; ++i)
        if (l + lanes * i < cols) p[l + lanes * i] = to_elem<T>(v[i]);
    }
  }

  // Codes of the held columns f under the scale 2^e.
  static __device__ __forceinline__ void encode(uint8_t* __restrict__ codes, int l, int cols, const float (&f)[n], int e) {
    const float inv = pow2f(-e);
    uint32_t w[n / 4];
#pragma unroll
    for (int i = 0; i < n / 4; ++i)
      w[i] = e4m3x2(f[4 * i] * inv, f[4 * i + 1] * inv) | e4m3x2(f[4 * i + 2] * inv, f[4 * i + 3] * inv) << 16;
    if (e == kTopExponent) {  // 256 (0x78) becomes 240 (0x77), four codes at once
#pragma unroll
      for (int i = 0; i < n / 4; ++i) w[i] -= __vcmpeq4(w[i] & 0x7f7f7f7fu, 0x78787878u) & 0x01010101u;
    }
    if constexpr (kVec) {
#pragma unroll
      for (int c = 0; c < chunks; ++c)
        if (chunk(l, c) < cols) *reinterpret_cast<uint2*>(codes + chunk(l, c)) = make_uint2(w[2 * c], w[2 * c + 1]);
    } else {
#pragma unroll
      for (int i = 0; i < n; ++i)
        if (l + lanes * i < cols) codes[l + lanes * i] = (uint8_t)(w[i / 4] >> (8 * (i % 4)));
    }
  }

  static __device__ __forceinline__ void load_codes(const uint8_t* __restrict__ codes, int l, int cols, uint32_t (&w)[n / 4]) {
    if constexpr (kVec) {
#pragma unroll
      for (int c = 0; c < chunks; ++c) {
        const int at = chunk(l, c);
        const uint2 v = at < cols ? __ldg(reinterpret_cast<const uint2*>(codes + at)) : make_uint2(0u, 0u);
        w[2 * c] = v.x, w[2 * c + 1] = v.y;
      }
    } else {
      uint32_t c[n];
#pragma unroll
      for (int i = 0; i < n; ++i) c[i] = l + lanes * i < cols ? __ldg(codes + l + lanes * i) : 0u;
#pragma unroll
      for (int i = 0; i < n / 4; ++i) w[i] = c[4 * i] | c[4 * i + 1] << 8 | c[4 * i + 2] << 16 | c[4 * i + 3] << 24;
    }
  }

  static __device__ __forceinline__ void decode(const uint32_t (&w)[n / 4], float scale, float (&v)[n]) {
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
      const float2 f = e4m3x2_values(w[i / 2] >> (16 * (i & 1)));
      v[2 * i] = f.x * scale;
      v[2 * i + 1] = f.y * scale;
    }
  }
};

// Lanes per block where columns are taken one by one.
constexpr int kForwardLanes = 16, kBackwardLanes = 32;

// One block of a matrix with per_row blocks of 128 columns per row and `total`
// blocks in all (below 2^30, so that 32-bit divisions find it).
struct Blocks {
  uint32_t total, per_row;
};
struct Block {
  int64_t row;
  uint32_t i;  // block of the row
  int n;       // its columns; 0 past the last block
};
__device__ __forceinline__ Block block_at(const Blocks& blk, uint32_t b, int64_t width) {
  Block o;
  const uint32_t row = b / blk.per_row;
  o.row = row;
  o.i = b - row * blk.per_row;
  o.n = b < blk.total ? (int)min((int64_t)128, width - (int64_t)o.i * 128) : 0;
  return o;
}

// This thread's block; every thread of a warp goes on whatever its block is (it
// holds no columns past the last), so that the shuffles are whole.
template <int lanes>
__device__ __forceinline__ uint32_t own_block() {
  return (uint32_t)(((uint64_t)blockIdx.x * kThreads + threadIdx.x) / lanes);
}

// HBM-bound: 32768 x 4096 bf16 in 58 us (6.9 TB/s).
template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads)
    checkpoint_kernel(const T* __restrict__ x, Blocks blk, int64_t K, int64_t ld, uint8_t* __restrict__ codes,
                      float* __restrict__ scales, int* status) {
  pdl_wait();
  using H = Held<T, kVec, kForwardLanes>;
  const int l = threadIdx.x & (H::lanes - 1);
  const uint32_t b = own_block<H::lanes>();
  const Block k = block_at(blk, b, K);
  const int64_t c = (int64_t)k.i * 128;
  H v;
  v.load(x + k.row * ld + c, l, k.n);
  const float top = v.amax();
  const int e = scale_exponent(top);
  float f[H::n];
  v.floats(f);
  H::encode(codes + k.row * K + c, l, k.n, f, e);
  if (l == 0 && k.n > 0) {
    scales[b] = pow2f(e);
    if (nonfinite(top)) latch_status(status, Q4_ERR_NONFINITE);
  }
}

// One pass: both halves' checkpoints and h.  HBM-bound: 32768 x 2 x 2048 bf16 in
// 79 us (6.8 TB/s).
template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads)
    swiglu_kernel(const T* __restrict__ gate_up, Blocks blk, int64_t I, int64_t ld, T* __restrict__ h,
                  uint8_t* __restrict__ codes, float* __restrict__ scales, int* status) {
  pdl_wait();
  using H = Held<T, kVec, kForwardLanes>;
  const int l = threadIdx.x & (H::lanes - 1);
  const Block k = block_at(blk, own_block<H::lanes>(), I);
  const int64_t c = (int64_t)k.i * 128;
  H hg, hu;
  hg.load(gate_up + k.row * ld + c, l, k.n);
  hu.load(gate_up + k.row * ld + I + c, l, k.n);
  const float tg = hg.amax(), tu = hu.amax();
  const int eg = scale_exponent(tg), eu = scale_exponent(tu);
  float g[H::n], u[H::n];
  hg.floats(g);
  hu.floats(u);
  H::encode(codes + k.row * 2 * I + c, l, k.n, g, eg);
  H::encode(codes + k.row * 2 * I + I + c, l, k.n, u, eu);
  if (l == 0 && k.n > 0) {
    scales[k.row * 2 * blk.per_row + k.i] = pow2f(eg);
    scales[k.row * 2 * blk.per_row + blk.per_row + k.i] = pow2f(eu);
    if (nonfinite(tg) || nonfinite(tu)) latch_status(status, Q4_ERR_NONFINITE);
  }
#pragma unroll
  for (int j = 0; j < H::n; ++j) g[j] = g[j] * sigmoid(g[j]) * u[j];
  H::store(h + k.row * I + c, l, k.n, g);
}

// HBM-bound: 32768 x 2048 bf16 in 77 us (6.9 TB/s); columns one by one 9973 x 1411
// in 27 us (4.2 TB/s).
template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads)
    swiglu_backward_kernel(const T* __restrict__ d_h, Blocks blk, int64_t I, int64_t ld,
                           const uint8_t* __restrict__ codes, const float* __restrict__ scales,
                           T* __restrict__ d_gate_up) {
  pdl_wait();
  using H = Held<T, kVec, kBackwardLanes>;
  const int l = threadIdx.x & (H::lanes - 1);
  const uint32_t b = own_block<H::lanes>();
  if (b >= blk.total) return;
  const Block k = block_at(blk, b, I);
  const int64_t c = (int64_t)k.i * 128;
  const float* sc = scales + k.row * 2 * blk.per_row + k.i;
  uint32_t wg[H::n / 4], wu[H::n / 4];
  H hd;
  hd.load(d_h + k.row * ld + c, l, k.n);
  H::load_codes(codes + k.row * 2 * I + c, l, k.n, wg);
  H::load_codes(codes + k.row * 2 * I + I + c, l, k.n, wu);
  const float sg = __ldg(sc), su = __ldg(sc + blk.per_row);
  float g[H::n], u[H::n], d[H::n];
  H::decode(wg, sg, g);
  H::decode(wu, su, u);
  hd.floats(d);
#pragma unroll
  for (int j = 0; j < H::n; ++j) {
    const float s = sigmoid(g[j]);
    const float ds = d[j] * s, du = ds * g[j];
    g[j] = ds * u[j] * fmaf(g[j], 1.f - s, 1.f);
    u[j] = du;
  }
  H::store(d_gate_up + k.row * 2 * I + c, l, k.n, g);
  H::store(d_gate_up + k.row * 2 * I + I + c, l, k.n, u);
}

// One turn per thread: the blocks of threads are many and alike, and the
// hardware keeps the SMs full of them (a grid of 8 per SM that loops left the
// SMs 62% occupied at the end: 119 us instead of 93 at 32768 x 2 x 2048 bf16).
template <typename T, int kSingle>
unsigned block_grid(const Blocks& blk, bool vec) {
  return (unsigned)ceil_div(blk.total, kThreads / (vec ? Held<T, true, kSingle>::lanes : kSingle));
}

}  // namespace

q4_status launch_checkpoint(const void* x, int dtype, int64_t rows, int64_t K, int64_t ld, uint8_t* codes,
                            float* scales, cudaStream_t stream) {
  const Blocks blk{(uint32_t)(rows * ceil_div(K, 128)), (uint32_t)ceil_div(K, 128)};
  return by_dtype(dtype, [&](auto tag) {
    using T = decltype(tag);
    const bool vec = K % 8 == 0 && ld * sizeof(T) % 16 == 0 && mult(x, 16) && mult(codes, 8);
    return launch_pdl(vec ? checkpoint_kernel<T, true> : checkpoint_kernel<T, false>, block_grid<T, kForwardLanes>(blk, vec), kThreads, 0,
                      stream, static_cast<const T*>(x), blk, K, ld, codes, scales, device_status_ptr());
  });
}

q4_status launch_swiglu(const void* gate_up, int dtype, int64_t rows, int64_t I, int64_t ld, void* h, uint8_t* codes,
                        float* scales, cudaStream_t stream) {
  const Blocks blk{(uint32_t)(rows * ceil_div(I, 128)), (uint32_t)ceil_div(I, 128)};
  return by_dtype(dtype, [&](auto tag) {
    using T = decltype(tag);
    const bool vec = I % 8 == 0 && ld * sizeof(T) % 16 == 0 && mult(gate_up, 16) && mult(h, 16) && mult(codes, 8);
    return launch_pdl(vec ? swiglu_kernel<T, true> : swiglu_kernel<T, false>, block_grid<T, kForwardLanes>(blk, vec), kThreads, 0, stream,
                      static_cast<const T*>(gate_up), blk, I, ld, static_cast<T*>(h), codes, scales,
                      device_status_ptr());
  });
}

q4_status launch_swiglu_backward(const void* d_h, int dtype, int64_t rows, int64_t I, int64_t ld,
                                 const uint8_t* codes, const float* scales, void* d_gate_up, cudaStream_t stream) {
  const Blocks blk{(uint32_t)(rows * ceil_div(I, 128)), (uint32_t)ceil_div(I, 128)};
  return by_dtype(dtype, [&](auto tag) {
    using T = decltype(tag);
    const bool vec = I % 8 == 0 && ld * sizeof(T) % 16 == 0 && mult(d_h, 16) && mult(codes, 8) && mult(d_gate_up, 16);
    return launch_pdl(vec ? swiglu_backward_kernel<T, true> : swiglu_backward_kernel<T, false>, block_grid<T, kBackwardLanes>(blk, vec),
                      kThreads, 0, stream, static_cast<const T*>(d_h), blk, I, ld, codes, scales,
                      static_cast<T*>(d_gate_up));
  });
}

}  // namespace q4
