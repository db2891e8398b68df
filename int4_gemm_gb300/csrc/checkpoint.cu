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
// even).
//
// swiglu of gate_up = [g | u]:  h = silu(g) u,  silu(g) = g / (1 + exp(-g));
// its gradient at the restored g and u, with s = 1 / (1 + exp(-g)):
//   dg = dh u s (1 + g (1 - s)),  du = dh g s.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "quant_device.cuh"

namespace q4 {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// The values of the two codes in the low 16 bits.
__device__ __forceinline__ float2 e4m3x2_values(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Exponent of the block's scale: 448 = 1.75 * 2^8, so the significand of amax
// decides between its own exponent - 8 and - 7.
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t b = __float_as_uint(fmaxf(amax, 1e-12f));
  return (int)((b + 0x1fffffu) >> 23) - 127 - 8;
}
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

template <typename T>
__device__ __forceinline__ T to_elem(float v);
template <>
__device__ __forceinline__ float to_elem<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 to_elem<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half to_elem<__half>(float v) { return __float2half_rn(v); }

// silu's factor 1 / (1 + exp(-g)) with the fast exponential and reciprocal
// (below 2^-17 relative error for |g| <= 88; below g = -87.3 it is 0 instead
// of less than 1e-37).  The exact functions cost more issue slots than the
// whole rest of the kernels.
__device__ __forceinline__ float sigmoid(float g) { return __fdividef(1.f, 1.f + __expf(-g)); }

// A half-warp holds one block of 128 columns, 8 per lane: columns 8 l .. of
// lane l with 128-bit accesses (kVec), or l, l + 16, ... one by one, the ones
// past the block's end as zeros.
template <typename T, bool kVec>
__device__ __forceinline__ void load_block(const T* __restrict__ p, int l, int n, float (&v)[8]) {
  if constexpr (kVec) {
    if (8 * l < n) {
      load8<T>(p, 8 * l, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = l + 16 * i < n ? Elem<T>::to_f(p[l + 16 * i]) : 0.f;
  }
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

template <typename T, bool kVec>
__device__ __forceinline__ void store_block(T* __restrict__ p, int l, int n, const float (&v)[8]) {
  if constexpr (kVec) {
    if (8 * l < n) {
      uint4* out = reinterpret_cast<uint4*>(p + 8 * l);
      if constexpr (sizeof(T) == 4) {
        out[0] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
        out[1] = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
      } else {
        out[0] = make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (l + 16 * i < n) p[l + 16 * i] = to_elem<T>(v[i]);
  }
}

// Codes of one block; returns its scale (the same in all 16 lanes).  The
// largest magnitude is taken on the bit patterns, where NaN and infinity come
// out on top and need no test of their own.
template <bool kVec>
__device__ __forceinline__ float encode_block(uint8_t* __restrict__ codes, int l, int n, const float (&v)[8],
                                              bool& bad) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  bad |= top >= 0x7f800000u;
  const int e = min(scale_exponent(__uint_as_float(top)), 120);
  const float inv = pow2f(-e);
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    w[i] = e4m3x2(v[4 * i] * inv, v[4 * i + 1] * inv) | e4m3x2(v[4 * i + 2] * inv, v[4 * i + 3] * inv) << 16;
  if constexpr (kVec) {
    if (8 * l < n) *reinterpret_cast<uint2*>(codes + 8 * l) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (l + 16 * i < n) codes[l + 16 * i] = (uint8_t)(w[i / 4] >> (8 * (i % 4)));
  }
  return pow2f(e);
}

template <bool kVec>
__device__ __forceinline__ void decode_block(const uint8_t* __restrict__ codes, float scale, int l, int n,
                                             float (&v)[8]) {
  uint32_t w[2] = {0u, 0u};
  if constexpr (kVec) {
    if (8 * l < n) {
      const uint2 c = __ldg(reinterpret_cast<const uint2*>(codes + 8 * l));
      w[0] = c.x, w[1] = c.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (l + 16 * i < n) w[i / 4] |= (uint32_t)codes[l + 16 * i] << (8 * (i % 4));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = e4m3x2_values(w[i / 2] >> (16 * (i & 1)));
    v[2 * i] = f.x * scale;
    v[2 * i + 1] = f.y * scale;
  }
}

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

// Both half-warps of a warp take the same number of turns, so that the
// shuffles stay whole.
template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads)
    checkpoint_kernel(const T* __restrict__ x, Blocks blk, int64_t K, int64_t ld, uint8_t* __restrict__ codes,
                      float* __restrict__ scales, int* status) {
  pdl_wait();
  const int l = threadIdx.x & 15;
  bool bad = false;
  for (uint32_t b0 = (blockIdx.x * kThreads + threadIdx.x) / 32 * 2; b0 < blk.total; b0 += gridDim.x * (kThreads / 16)) {
    const uint32_t b = b0 + (threadIdx.x >> 4 & 1);
    const Block k = block_at(blk, b, K);
    const int64_t c = (int64_t)k.i * 128;
    float v[8];
    load_block<T, kVec>(x + k.row * ld + c, l, k.n, v);
    const float s = encode_block<kVec>(codes + k.row * K + c, l, k.n, v, bad);
    if (l == 0 && k.n > 0) scales[b] = s;
  }
  if (__any_sync(0xffffffffu, bad) && (threadIdx.x & 31) == 0) latch_status(status, Q4_ERR_NONFINITE);
}

template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads)
    swiglu_kernel(const T* __restrict__ gate_up, Blocks blk, int64_t I, int64_t ld, T* __restrict__ h,
                  uint8_t* __restrict__ codes, float* __restrict__ scales, int* status) {
  pdl_wait();
  const int l = threadIdx.x & 15;
  bool bad = false;
  for (uint32_t b0 = (blockIdx.x * kThreads + threadIdx.x) / 32 * 2; b0 < blk.total; b0 += gridDim.x * (kThreads / 16)) {
    const Block k = block_at(blk, b0 + (threadIdx.x >> 4 & 1), I);
    const int64_t c = (int64_t)k.i * 128;
    float g[8], u[8];
    load_block<T, kVec>(gate_up + k.row * ld + c, l, k.n, g);
    load_block<T, kVec>(gate_up + k.row * ld + I + c, l, k.n, u);
    const float sg = encode_block<kVec>(codes + k.row * 2 * I + c, l, k.n, g, bad);
    const float su = encode_block<kVec>(codes + k.row * 2 * I + I + c, l, k.n, u, bad);
    if (l == 0 && k.n > 0) {
      scales[k.row * 2 * blk.per_row + k.i] = sg;
      scales[k.row * 2 * blk.per_row + blk.per_row + k.i] = su;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = g[j] * sigmoid(g[j]) * u[j];
    store_block<T, kVec>(h + k.row * I + c, l, k.n, g);
  }
  if (__any_sync(0xffffffffu, bad) && (threadIdx.x & 31) == 0) latch_status(status, Q4_ERR_NONFINITE);
}

template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads)
    swiglu_backward_kernel(const T* __restrict__ d_h, Blocks blk, int64_t I, int64_t ld,
                           const uint8_t* __restrict__ codes, const float* __restrict__ scales,
                           T* __restrict__ d_gate_up) {
  pdl_wait();
  const int l = threadIdx.x & 15;
  for (uint32_t b = (blockIdx.x * kThreads + threadIdx.x) / 16; b < blk.total; b += gridDim.x * (kThreads / 16)) {
    const Block k = block_at(blk, b, I);
    const int64_t c = (int64_t)k.i * 128;
    const float* sc = scales + k.row * 2 * blk.per_row + k.i;
    float g[8], u[8], d[8];
    load_block<T, kVec>(d_h + k.row * ld + c, l, k.n, d);
    decode_block<kVec>(codes + k.row * 2 * I + c, __ldg(sc), l, k.n, g);
    decode_block<kVec>(codes + k.row * 2 * I + I + c, __ldg(sc + blk.per_row), l, k.n, u);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float s = sigmoid(g[j]);
      const float ds = d[j] * s, du = ds * g[j];
      g[j] = ds * u[j] * fmaf(g[j], 1.f - s, 1.f);
      u[j] = du;
    }
    store_block<T, kVec>(d_gate_up + k.row * 2 * I + c, l, k.n, g);
    store_block<T, kVec>(d_gate_up + k.row * 2 * I + I + c, l, k.n, u);
  }
}

template <typename F>
q4_status by_dtype(int dtype, F&& f) {
  if (dtype == Q4_F32) return f(float());
  if (dtype == Q4_BF16) return f(__nv_bfloat16());
  return f(__half());
}

inline bool mult(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

unsigned block_grid(const Blocks& blk) {
  return (unsigned)std::min<int64_t>(ceil_div(blk.total, kThreads / 16), (int64_t)num_sms() * 8);
}

}  // namespace

q4_status launch_checkpoint(const void* x, int dtype, int64_t rows, int64_t K, int64_t ld, uint8_t* codes,
                            float* scales, cudaStream_t stream) {
  const Blocks blk{(uint32_t)(rows * ceil_div(K, 128)), (uint32_t)ceil_div(K, 128)};
  return by_dtype(dtype, [&](auto tag) {
    using T = decltype(tag);
    const bool vec = K % 8 == 0 && ld * sizeof(T) % 16 == 0 && mult(x, 16) && mult(codes, 8);
    return launch_pdl(vec ? checkpoint_kernel<T, true> : checkpoint_kernel<T, false>, block_grid(blk), kThreads, 0,
                      stream, static_cast<const T*>(x), blk, K, ld, codes, scales, device_status_ptr());
  });
}

q4_status launch_swiglu(const void* gate_up, int dtype, int64_t rows, int64_t I, int64_t ld, void* h, uint8_t* codes,
                        float* scales, cudaStream_t stream) {
  const Blocks blk{(uint32_t)(rows * ceil_div(I, 128)), (uint32_t)ceil_div(I, 128)};
  return by_dtype(dtype, [&](auto tag) {
    using T = decltype(tag);
    const bool vec = I % 8 == 0 && ld * sizeof(T) % 16 == 0 && mult(gate_up, 16) && mult(h, 16) && mult(codes, 8);
    return launch_pdl(vec ? swiglu_kernel<T, true> : swiglu_kernel<T, false>, block_grid(blk), kThreads, 0, stream,
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
    return launch_pdl(vec ? swiglu_backward_kernel<T, true> : swiglu_backward_kernel<T, false>, block_grid(blk),
                      kThreads, 0, stream, static_cast<const T*>(d_h), blk, I, ld, codes, scales,
                      static_cast<T*>(d_gate_up));
  });
}

}  // namespace q4
