// Weight gradient of routed experts from 8-bit activation checkpoints:
//   dW[e] (+)= sum over the rows r of expert e of d_y[r]^T x[row_token[r]],
//   x = bf16(codes * scales) (E4M3, one scale per row and 128 columns; exact
//   for the power-of-two scales of a checkpoint), bf16 d_y.
// Products are formed in FP32 and summed over the expert's rows in order.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace q4 {
namespace {

constexpr int kTile = 64, kRows = 16, kThreads = 256;

__device__ __forceinline__ float e4m3_to_f(uint8_t code) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)code));
  return __half2float(__ushort_as_half((uint16_t)h));
}

// One 64 x 64 tile of dW[blockIdx.z] per block, 4 x 4 outputs per thread,
// sixteen rows staged in shared memory at a time.
template <typename W>
__global__ void __launch_bounds__(kThreads)
    wgrad_simple_kernel(const __nv_bfloat16* __restrict__ dy, int64_t R, int64_t N, int64_t ldy,
                        const uint8_t* __restrict__ codes, const float* __restrict__ scales, int64_t tokens,
                        int64_t K, const int32_t* __restrict__ row_token, const int32_t* __restrict__ offsets,
                        W* __restrict__ dw, int accumulate) {
  pdl_wait();
  __shared__ float a[kRows][kTile], b[kRows][kTile];
  const int64_t n0 = (int64_t)blockIdx.y * kTile, k0 = (int64_t)blockIdx.x * kTile, e = blockIdx.z;
  const int64_t KB = (K + 127) / 128;
  const int64_t lo = max((int64_t)__ldg(offsets + e), (int64_t)0), hi = min((int64_t)__ldg(offsets + e + 1), R);
  const int tn = threadIdx.x / 16 * 4, tk = threadIdx.x % 16 * 4;
  float acc[4][4] = {};
  for (int64_t r0 = lo; r0 < hi; r0 += kRows) {
    for (int i = threadIdx.x; i < kRows * kTile; i += kThreads) {
      const int64_t r = r0 + i / kTile, n = n0 + i % kTile, k = k0 + i % kTile;
      float va = 0.f, vb = 0.f;
      if (r < hi) {
        if (n < N) va = __bfloat162float(dy[r * ldy + n]);
        const int64_t t = row_token ? __ldg(row_token + r) : r;
        if (k < K && t >= 0 && t < tokens) vb = __bfloat162float(__float2bfloat16_rn(e4m3_to_f(codes[t * K + k]) * __ldg(scales + t * KB + k / 128)));
      }
      a[i / kTile][i % kTile] = va;
      b[i / kTile][i % kTile] = vb;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[r][tn + i], b[r][tk + j], acc[i][j]);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t n = n0 + tn + i, k = k0 + tk + j;
      if (n >= N || k >= K) continue;
      W* out = dw + (e * N + n) * K + k;
      if constexpr (sizeof(W) == 4)
        *out = accumulate ? *out + acc[i][j] : acc[i][j];
      else
        *out = __float2bfloat16_rn(acc[i][j]);
    }
}

}  // namespace

size_t wgrad_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

q4_status launch_wgrad(const WgradArgs& a, cudaStream_t stream) {
  const dim3 grid((unsigned)ceil_div(a.K, kTile), (unsigned)ceil_div(a.N, kTile), (unsigned)a.E);
  const __nv_bfloat16* dy = static_cast<const __nv_bfloat16*>(a.dy);
  if (a.w_dtype == Q4_F32)
    return launch_pdl(wgrad_simple_kernel<float>, grid, kThreads, 0, stream, dy, a.R, a.N, a.ldy, a.codes, a.scales,
                      a.tokens, a.K, a.row_token, a.offsets, static_cast<float*>(a.dw), (int)a.accumulate);
  return launch_pdl(wgrad_simple_kernel<__nv_bfloat16>, grid, kThreads, 0, stream, dy, a.R, a.N, a.ldy, a.codes,
                    a.scales, a.tokens, a.K, a.row_token, a.offsets, static_cast<__nv_bfloat16*>(a.dw), 0);
}

}  // namespace q4
