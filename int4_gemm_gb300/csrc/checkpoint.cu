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
__device__ __forceinline__ float e4m3_value(uint32_t code) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)code));
  return __half2float(__ushort_as_half((uint16_t)h));
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

// A half-warp holds one block of 128 columns, 8 per lane: columns 8 l .. of
// lane l with 128-bit accesses (kVec), or l, l + 16, ... one by one, the ones
// past the block's end as zeros.
template <bool kVec>
__device__ __forceinline__ int column(int lane16, int i) { return kVec ? lane16 * 8 + i : lane16 + 16 * i; }

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
    for (int i = 0; i < 8; ++i) v[i] = column<false>(l, i) < n ? Elem<T>::to_f(p[column<false>(l, i)]) : 0.f;
  }
}

template <typename T, bool kVec>
__device__ __forceinline__ void store_block(T* __restrict__ p, int l, int n, const float (&v)[8]) {
  if constexpr (kVec) {
    if (8 * l < n) {
      __align__(16) T o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = to_elem<T>(v[i]);
#pragma unroll
      for (int i = 0; i < (int)sizeof(o) / 16; ++i)
        reinterpret_cast<uint4*>(p + 8 * l)[i] = reinterpret_cast<const uint4*>(o)[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (column<false>(l, i) < n) p[column<false>(l, i)] = to_elem<T>(v[i]);
  }
}

// Codes of one block; returns its scale (the same in all 16 lanes).
template <bool kVec>
__device__ __forceinline__ float encode_block(uint8_t* __restrict__ codes, int l, int n, const float (&v)[8],
                                              bool& bad) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    bad |= nonfinite(v[i]);
    amax = fmaxf(amax, fabsf(v[i]));
  }
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const int e = min(scale_exponent(amax), 120);
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
      if (column<false>(l, i) < n) codes[column<false>(l, i)] = (uint8_t)(w[i / 4] >> (8 * (i % 4)));
  }
  return pow2f(e);
}

template <bool kVec>
__device__ __forceinline__ void decode_block(const uint8_t* __restrict__ codes, float scale, int l, int n,
                                             float (&v)[8]) {
  if constexpr (kVec) {
    uint2 w = make_uint2(0u, 0u);
    if (8 * l < n) w = __ldg(reinterpret_cast<const uint2*>(codes + 8 * l));
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = e4m3_value((i < 4 ? w.x : w.y) >> (8 * (i % 4)) & 0xffu) * scale;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = column<false>(l, i) < n ? e4m3_value(codes[column<false>(l, i)]) * scale : 0.f;
  }
}

// Block index of this half-warp, over all blocks of all rows; every lane of a
// warp takes the same number of turns so that the shuffles stay whole.
struct Blocks {
  int64_t total;
  int per_row;
};

template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads)
    checkpoint_kernel(const T* __restrict__ x, Blocks blk, int64_t K, int64_t ld, uint8_t* __restrict__ codes,
                      float* __restrict__ scales, int* status) {
  pdl_wait();
  const int l = threadIdx.x & 15;
  const int64_t step = (int64_t)gridDim.x * (kThreads / 16);
  bool bad = false;
  for (int64_t b0 = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / 32 * 2; b0 < blk.total; b0 += step) {
    const int64_t b = b0 + (threadIdx.x >> 4 & 1);
    const int64_t row = b / blk.per_row, c = (b - row * blk.per_row) * 128;
    const int n = b < blk.total ? (int)min((int64_t)128, K - c) : 0;
    float v[8];
    load_block<T, kVec>(x + row * ld + c, l, n, v);
    const float s = encode_block<kVec>(codes + row * K + c, l, n, v, bad);
    if (l == 0 && n > 0) scales[b] = s;
  }
  if (__any_sync(0xffffffffu, bad) && (threadIdx.x & 31) == 0) latch_status(status, Q4_ERR_NONFINITE);
}

template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads)
    swiglu_kernel(const T* __restrict__ gate_up, Blocks blk, int64_t I, int64_t ld, T* __restrict__ h,
                  uint8_t* __restrict__ codes, float* __restrict__ scales, int* status) {
  pdl_wait();
  const int l = threadIdx.x & 15;
  const int64_t step = (int64_t)gridDim.x * (kThreads / 16);
  bool bad = false;
  for (int64_t b0 = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / 32 * 2; b0 < blk.total; b0 += step) {
    const int64_t b = b0 + (threadIdx.x >> 4 & 1);
    const int64_t row = b / blk.per_row, i = b - row * blk.per_row, c = i * 128;
    const int n = b < blk.total ? (int)min((int64_t)128, I - c) : 0;
    float g[8], u[8];
    load_block<T, kVec>(gate_up + row * ld + c, l, n, g);
    load_block<T, kVec>(gate_up + row * ld + I + c, l, n, u);
    const float sg = encode_block<kVec>(codes + row * 2 * I + c, l, n, g, bad);
    const float su = encode_block<kVec>(codes + row * 2 * I + I + c, l, n, u, bad);
    if (l == 0 && n > 0) {
      scales[row * 2 * blk.per_row + i] = sg;
      scales[row * 2 * blk.per_row + blk.per_row + i] = su;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = g[j] / (1.f + expf(-g[j])) * u[j];
    store_block<T, kVec>(h + row * I + c, l, n, g);
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
  const int64_t step = (int64_t)gridDim.x * (kThreads / 16);
  for (int64_t b = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / 16; b < blk.total; b += step) {
    const int64_t row = b / blk.per_row, i = b - row * blk.per_row, c = i * 128;
    const int n = (int)min((int64_t)128, I - c);
    const float* sc = scales + row * 2 * blk.per_row + i;
    float g[8], u[8], d[8];
    decode_block<kVec>(codes + row * 2 * I + c, __ldg(sc), l, n, g);
    decode_block<kVec>(codes + row * 2 * I + I + c, __ldg(sc + blk.per_row), l, n, u);
    load_block<T, kVec>(d_h + row * ld + c, l, n, d);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float s = 1.f / (1.f + expf(-g[j]));
      const float du = d[j] * g[j] * s;
      g[j] = d[j] * u[j] * s * (1.f + g[j] * (1.f - s));
      u[j] = du;
    }
    store_block<T, kVec>(d_gate_up + row * 2 * I + c, l, n, g);
    store_block<T, kVec>(d_gate_up + row * 2 * I + I + c, l, n, u);
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
  const Blocks blk{rows * ceil_div(K, 128), (int)ceil_div(K, 128)};
  return by_dtype(dtype, [&](auto tag) {
    using T = decltype(tag);
    const bool vec = K % 8 == 0 && ld * sizeof(T) % 16 == 0 && mult(x, 16) && mult(codes, 8);
    return launch_pdl(vec ? checkpoint_kernel<T, true> : checkpoint_kernel<T, false>, block_grid(blk), kThreads, 0,
                      stream, static_cast<const T*>(x), blk, K, ld, codes, scales, device_status_ptr());
  });
}

q4_status launch_swiglu(const void* gate_up, int dtype, int64_t rows, int64_t I, int64_t ld, void* h, uint8_t* codes,
                        float* scales, cudaStream_t stream) {
  const Blocks blk{rows * ceil_div(I, 128), (int)ceil_div(I, 128)};
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
  const Blocks blk{rows * ceil_div(I, 128), (int)ceil_div(I, 128)};
  return by_dtype(dtype, [&](auto tag) {
    using T = decltype(tag);
    const bool vec = I % 8 == 0 && ld * sizeof(T) % 16 == 0 && mult(d_h, 16) && mult(codes, 8) && mult(d_gate_up, 16);
    return launch_pdl(vec ? swiglu_backward_kernel<T, true> : swiglu_backward_kernel<T, false>, block_grid(blk),
                      kThreads, 0, stream, static_cast<const T*>(d_h), blk, I, ld, codes, scales,
                      static_cast<T*>(d_gate_up));
  });
}

}  // namespace q4
