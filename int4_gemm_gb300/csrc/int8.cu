// 8-bit integers with one scale per row: the quantizer and the product
//   C[m, n] = sa[m] sb[n] sum over k of qa[m, k] qb[n, k]
// with exact 32-bit integer sums.
//
// The quantizer follows the oracle step by step in FP32 with IEEE rounding:
//   s = max(amax, 1e-12) / 127,  q = rint(x / s)  (ties to even)
#include <algorithm>

#include "common.cuh"
#include "elem.cuh"
#include "internal.h"

namespace q4 {
namespace {

constexpr int kQuantThreads = 256;

// One block of threads per row: the largest magnitude, then the codes (the row
// comes from L1 or L2 the second time).
template <typename T>
__global__ void __launch_bounds__(kQuantThreads)
    quantize_int8_kernel(const T* __restrict__ x, int64_t K, int64_t ld, int8_t* __restrict__ codes, float* __restrict__ scales,
                         int* status) {
  pdl_wait();
  __shared__ uint32_t part[kQuantThreads / 32];
  const T* row = x + (int64_t)blockIdx.x * ld;
  uint32_t top = 0;  // as bits: NaN and infinities come out on top
  for (int64_t k = threadIdx.x; k < K; k += kQuantThreads) top = max(top, __float_as_uint(Elem<T>::to_f(row[k])) & 0x7fffffffu);
  top = __reduce_max_sync(0xffffffffu, top);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = top;
  __syncthreads();
  for (int w = 0; w < kQuantThreads / 32; ++w) top = max(top, part[w]);
  const float s = __fdiv_rn(fmaxf(__uint_as_float(top), 1e-12f), 127.f);
  if (threadIdx.x == 0) {
    scales[blockIdx.x] = s;
    if (nonfinite(__uint_as_float(top))) latch_status(status, Q4_ERR_NONFINITE);
  }
  for (int64_t k = threadIdx.x; k < K; k += kQuantThreads)
    codes[(int64_t)blockIdx.x * K + k] = (int8_t)min(max(__float2int_rn(__fdiv_rn(Elem<T>::to_f(row[k]), s)), -127), 127);
}

// ------------------------------------------------------------------ product
constexpr int kTile = 64, kStep = 64, kPitch = kStep + 16;  // C tile, K bytes per stage, row pitch in shared memory

__device__ __forceinline__ void mma_s8(int (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <typename C>
__global__ void __launch_bounds__(128)
    int8_gemm_kernel(const int8_t* __restrict__ qa, const float* __restrict__ sa, const int8_t* __restrict__ qb,
                     const float* __restrict__ sb, int64_t M, int64_t N, int64_t K, C* __restrict__ out) {
  pdl_wait();
  __shared__ __align__(16) uint8_t ta[kTile * kPitch], tb[kTile * kPitch];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
  const int64_t m0 = (int64_t)blockIdx.x * kTile, n0 = (int64_t)blockIdx.y * kTile;
  int acc[8][4] = {};
  for (int64_t k0 = 0; k0 < K; k0 += kStep) {
    for (int i = threadIdx.x; i < kTile * kStep / 16; i += 128) {
      const int r = i / (kStep / 16), c = i % (kStep / 16) * 16;
      const bool in = k0 + c < K;
      const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
      *reinterpret_cast<uint4*>(ta + r * kPitch + c) =
          in && m0 + r < M ? *reinterpret_cast<const uint4*>(qa + (m0 + r) * K + k0 + c) : zero;
      *reinterpret_cast<uint4*>(tb + r * kPitch + c) =
          in && n0 + r < N ? *reinterpret_cast<const uint4*>(qb + (n0 + r) * K + k0 + c) : zero;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kStep; k += 32) {
      uint32_t a[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        a[i] = *reinterpret_cast<const uint32_t*>(ta + (warp * 16 + g + (i & 1) * 8) * kPitch + k + 4 * q + (i >> 1) * 16);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint8_t* b = tb + (j * 8 + g) * kPitch + k + 4 * q;
        mma_s8(acc[j], a, *reinterpret_cast<const uint32_t*>(b), *reinterpret_cast<const uint32_t*>(b + 16));
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t m = m0 + warp * 16 + g + (i >> 1) * 8, n = n0 + j * 8 + 2 * q + (i & 1);
      if (m < M && n < N) out[m * N + n] = to_elem<C>((float)acc[j][i] * sa[m] * sb[n]);
    }
}

}  // namespace

q4_status launch_quantize_int8(const void* x, int dtype, int64_t rows, int64_t K, int64_t ld, int8_t* codes, float* scales,
                               cudaStream_t stream) {
  return by_dtype(dtype, [&](auto tag) {
    using T = decltype(tag);
    return launch_pdl(quantize_int8_kernel<T>, (unsigned)rows, kQuantThreads, 0, stream, static_cast<const T*>(x), K, ld, codes,
                      scales, device_status_ptr());
  });
}

q4_status launch_int8_gemm(const int8_t* qa, const float* sa, const int8_t* qb, const float* sb, int64_t M, int64_t N, int64_t K,
                           void* C, int c_dtype, cudaStream_t stream) {
  const dim3 grid((unsigned)ceil_div(M, kTile), (unsigned)ceil_div(N, kTile));
  if (c_dtype == Q4_F32)
    return launch_pdl(int8_gemm_kernel<float>, grid, 128, 0, stream, qa, sa, qb, sb, M, N, K, static_cast<float*>(C));
  return launch_pdl(int8_gemm_kernel<__nv_bfloat16>, grid, 128, 0, stream, qa, sa, qb, sb, M, N, K, static_cast<__nv_bfloat16*>(C));
}

}  // namespace q4
