// 8-bit integers of a matrix, one scale per row, in FP32 steps with IEEE rounding as
// the oracle takes them:
//   s = max(amax, 1e-12) * RN(1 / 127),  q = rint(x / s)  (ties to even)
//
// HBM-bound: a row is read once and stays in registers (16 lanes per block of 128
// columns, rows.cuh), rows too long for that are read a second time from L2.
// x / s is taken as x * (1 / s), which is within 4 ulp of it, unless that lies within
// 2^-12 of a half-integer (a quotient below 128 is off by less than 2^-14), where it
// is divided.  8192 x 8192 bf16 49.1 us (4.1 TB/s: instruction issue, 58%; with a division
// for every element, single loads and two passes 62.6), 28672 x 8192 FP32 175 us (6.7
// TB/s), 100 x 7168 bf16 2.9 us.  Above 16384 columns, with single loads, the second
// pass and the division: 8192 x 28672 bf16 261 us (2.7 TB/s), FP32 323 (3.6 TB/s).
#include "rows.cuh"

namespace q4 {
namespace {

__device__ __forceinline__ int8_t quotient(float x, float s) {
  return (int8_t)min(max(__float2int_rn(__fdiv_rn(x, s)), -127), 127);
}

template <typename T, bool kVec, int kC>
__global__ void __launch_bounds__(max_threads(kC))
    quantize_int8_kernel(const T* __restrict__ x, int64_t rows, int width, int64_t ld, int8_t* __restrict__ codes,
                         float* __restrict__ scales, int group, int* status) {
  pdl_wait();
  using P = Piece<T, kVec>;
  __shared__ Exchange ex;
  exchange_init(ex);
  __syncthreads();
  const Place pl(group);
  int buf = 0;
  for (int64_t base = (int64_t)blockIdx.x * pl.per_block; base < rows; base += (int64_t)gridDim.x * pl.per_block, buf ^= 1) {
    const int64_t row = base + pl.sub;
    const int H = row < rows ? width : 0;
    P p[kC];
#pragma unroll
    for (int i = 0; i < kC; ++i) p[i].load(x + row * ld + pl.at(i), pl.l, pl.cols(i, H));
    uint32_t bits = 0;  // of magnitudes, pairs of 16-bit ones in a word: NaN and infinities come out on top
#pragma unroll
    for (int i = 0; i < kC; ++i)
#pragma unroll
      for (int j = 0; j < P::words; ++j) {
        if constexpr (P::packed)
          bits = __vmaxu2(bits, p[i].w[j] & 0x7fff7fffu);
        else
          bits = max(bits, p[i].w[j] & (sizeof(T) == 2 ? 0x7fffu : 0x7fffffffu));
      }
    if constexpr (P::packed) bits = max(bits >> 16, bits & 0xffffu);
    float top;
    if constexpr (sizeof(T) == 2)
      top = unpack2<T>(bits).x;
    else
      top = __uint_as_float(bits);
    const float2 r = group_reduce<true>(nonfinite(top) ? 1.f : 0.f, top, group, ex, buf);
    const float s = max_nan(r.y, 1e-12f) * (1.f / 127.f);
    if (pl.t == 0 && H) {
      scales[row] = s;
      if (r.x != 0.f) latch_status(status, Q4_ERR_NONFINITE);
    }
    const float inv = __fdividef(1.f, s);
    uint8_t* out = reinterpret_cast<uint8_t*>(codes) + row * width;
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      float v[8], far = 0.f;  // largest distance of a product from its integer
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] = p[i].at(j);
        const float q = __uint_as_float(int8_bits(v[j], inv)) - 12582912.f;
        far = fmaxf(far, fabsf(fmaf(v[j], inv, -q)));
      }
      uint2 c = int8x8(v, inv);
      if (far > 0.5f - 0x1p-12f) {
        uint32_t w[2] = {0u, 0u};
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j / 4] |= (uint32_t)(uint8_t)quotient(v[j], s) << (8 * (j % 4));
        c = make_uint2(w[0], w[1]);
      }
      P::store_codes(out + pl.at(i), pl.l, pl.cols(i, H), c);
    }
  }
}

// Rows of any length, a block of threads each.
constexpr int kLongThreads = 512;
template <typename T>
__global__ void __launch_bounds__(kLongThreads)
    quantize_int8_long_kernel(const T* __restrict__ x, int64_t K, int64_t ld, int8_t* __restrict__ codes,
                              float* __restrict__ scales, int* status) {
  pdl_wait();
  __shared__ uint32_t part[kLongThreads / 32];
  const T* row = x + (int64_t)blockIdx.x * ld;
  uint32_t top = 0;  // as bits: NaN and infinities come out on top
#pragma unroll 4
  for (int64_t k = threadIdx.x; k < K; k += kLongThreads) top = max(top, __float_as_uint(Elem<T>::to_f(row[k])) & 0x7fffffffu);
  top = __reduce_max_sync(0xffffffffu, top);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = top;
  __syncthreads();
  for (int w = 0; w < kLongThreads / 32; ++w) top = max(top, part[w]);
  const float s = max_nan(__uint_as_float(top), 1e-12f) * (1.f / 127.f);
  if (threadIdx.x == 0) {
    scales[blockIdx.x] = s;
    if (nonfinite(__uint_as_float(top))) latch_status(status, Q4_ERR_NONFINITE);
  }
#pragma unroll 4
  for (int64_t k = threadIdx.x; k < K; k += kLongThreads) codes[(int64_t)blockIdx.x * K + k] = quotient(Elem<T>::to_f(row[k]), s);
}

}  // namespace

q4_status launch_quantize_int8(const void* x, int dtype, int64_t rows, int64_t K, int64_t ld, int8_t* codes, float* scales,
                               cudaStream_t stream) {
  const int blocks = (int)std::min<int64_t>(ceil_div(K, 128), 1 << 20);
  return by_dtype(dtype, [&](auto tag) {
    using T = decltype(tag);
    const T* from = static_cast<const T*>(x);
    if (blocks > 128)
      return launch_pdl(quantize_int8_long_kernel<T>, (unsigned)rows, kLongThreads, 0, stream, from, K, ld, codes, scales,
                        device_status_ptr());
    const bool vec = K % 8 == 0 && ld * (int64_t)sizeof(T) % 16 == 0 && mult(x, 16) && mult(codes, 8);
    const int C = blocks <= 4 || (rows <= 2 * num_sms() && blocks <= 64) ? 1 : 4;
    const Shape s = spread(blocks, C, 256);
    const int grid = (int)std::min<int64_t>(ceil_div(rows, s.threads / s.group), (int64_t)num_sms() * std::max(1, 2048 / s.threads));
    auto launch = [&](auto kernel) {
      return launch_pdl(kernel, grid, s.threads, 0, stream, from, rows, (int)K, ld, codes, scales, s.group, device_status_ptr());
    };
    if (C == 1) return vec ? launch(quantize_int8_kernel<T, true, 1>) : launch(quantize_int8_kernel<T, false, 1>);
    return vec ? launch(quantize_int8_kernel<T, true, 4>) : launch(quantize_int8_kernel<T, false, 4>);
  });
}

}  // namespace q4
