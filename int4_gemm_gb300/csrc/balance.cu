// Balance loss of the router and its gradient.
//
//   p[t] = softmax(logits[t]) over the experts above -inf;  n: tokens with one
//   counts[e] = slots of expert e,  f[e] = counts[e] E / (n k)
//   P[e] = sum over t of p[t, e] / n,  loss = coeff sum over e of f[e] P[e]
//   d_logits[t, e] = d_loss coeff / n * p[t, e] (f[e] - sum over j of p[t, j] f[j])
// (counts are constants to the gradient).  Softmax and sums are FP32.
//
// A warp holds a token's logits, lane l the experts l, l + 32, ..., and adds its
// tokens' probabilities up in registers; the blocks' sums meet in the workspace
// and are added in a fixed order by a second kernel (the counts are integers,
// whose order does not matter).
#include <algorithm>

#include "common.cuh"
#include "elem.cuh"
#include "internal.h"

namespace q4 {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxExperts = 1024;
constexpr int kFinishThreads = 1024;

// A token's softmax in a warp: lane l holds experts l + 32 i.  NaN and +inf mask
// their expert; all zero (and false) where every expert is masked.
template <typename T, int kN>
__device__ __forceinline__ bool token_softmax(const T* __restrict__ row, int E, int lane, float (&p)[kN], bool& bad) {
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int e = lane + 32 * i;
    float v = e < E ? Elem<T>::to_f(row[e]) : -INFINITY;
    if (!(v < INFINITY)) {
      bad = true;
      v = -INFINITY;
    }
    p[i] = v;
    top = fmaxf(top, v);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (top == -INFINITY) {
#pragma unroll
    for (int i = 0; i < kN; ++i) p[i] = 0.f;
    return false;
  }
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    p[i] = __expf(p[i] - top);
    sum += p[i];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const float inv = __fdiv_rn(1.f, sum);
#pragma unroll
  for (int i = 0; i < kN; ++i) p[i] *= inv;
  return true;
}

template <typename T, int kN>
__global__ void __launch_bounds__(kThreads)
    balance_kernel(const T* __restrict__ logits, int64_t tokens, int E, int64_t ld, const int32_t* __restrict__ ids,
                   int64_t slots, float* __restrict__ part_p, int32_t* __restrict__ part_c, int* status) {
  pdl_wait();
  __shared__ float sum[kWarps][32 * kN];
  __shared__ int32_t count[kMaxExperts + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int e = threadIdx.x; e <= E; e += kThreads) count[e] = 0;
  __syncthreads();
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < slots; i += (int64_t)gridDim.x * kThreads) {
    const int e = __ldg(ids + i);
    if (e >= 0 && e < E) atomicAdd(&count[e], 1);
  }
  float acc[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) acc[i] = 0.f;
  int there = 0;
  bool bad = false;
  for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < tokens; t += (int64_t)gridDim.x * kWarps) {
    float p[kN];
    there += token_softmax<T, kN>(logits + t * ld, E, lane, p, bad);
#pragma unroll
    for (int i = 0; i < kN; ++i) acc[i] += p[i];
  }
  if (bad) latch_status(status, Q4_ERR_NONFINITE);
  if (lane == 0) atomicAdd(&count[E], there);
#pragma unroll
  for (int i = 0; i < kN; ++i) sum[warp][lane + 32 * i] = acc[i];
  __syncthreads();
  for (int e = threadIdx.x; e <= E; e += kThreads) {
    part_c[(int64_t)blockIdx.x * (E + 1) + e] = count[e];
    if (e == E) continue;
    float s = 0.f;
    for (int w = 0; w < kWarps; ++w) s += sum[w][e];
    part_p[(int64_t)blockIdx.x * E + e] = s;
  }
}

// f[e] from the counts (0 where no token takes part).
__device__ __forceinline__ float load_factor(int32_t count, int32_t n, int E, int top_k) {
  return n > 0 ? (float)count * ((float)E / ((float)n * (float)top_k)) : 0.f;
}

__global__ void __launch_bounds__(kFinishThreads)
    balance_finish_kernel(const float* __restrict__ part_p, const int32_t* __restrict__ part_c, int parts, int E,
                          int top_k, float coeff, float* __restrict__ loss, int32_t* __restrict__ counts,
                          float* __restrict__ mean) {
  pdl_wait();
  __shared__ int32_t tokens;
  __shared__ float warp_sum[kFinishThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (warp == 0) {
    int32_t n = 0;
    for (int q = lane; q < parts; q += 32) n += part_c[(int64_t)q * (E + 1) + E];
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    if (lane == 0) tokens = n, counts[E] = n;
  }
  __syncthreads();
  const int32_t n = tokens;
  float part = 0.f;
  for (int e = threadIdx.x; e < E; e += kFinishThreads) {
    int32_t c = 0;
    float s = 0.f;
    for (int q = 0; q < parts; ++q) {
      c += part_c[(int64_t)q * (E + 1) + e];
      s += part_p[(int64_t)q * E + e];
    }
    const float m = n > 0 ? __fdiv_rn(s, (float)n) : 0.f;
    counts[e] = c;
    mean[e] = m;
    part = fmaf(load_factor(c, n, E, top_k), m, part);
  }
  for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
  if (lane == 0) warp_sum[warp] = part;
  __syncthreads();
  if (threadIdx.x == 0) {
    float s = 0.f;
    for (int w = 0; w < kFinishThreads / 32; ++w) s += warp_sum[w];
    *loss = coeff * s;
  }
}

template <typename T, int kN>
__global__ void __launch_bounds__(kThreads)
    balance_backward_kernel(const T* __restrict__ logits, int64_t tokens, int E, int64_t ld, const int32_t* __restrict__ counts,
                            int top_k, const float* __restrict__ d_loss, float coeff, int accumulate, T* __restrict__ d_logits) {
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t n = __ldg(counts + E);
  const float g = n > 0 ? __ldg(d_loss) * __fdiv_rn(coeff, (float)n) : 0.f;
  float f[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) f[i] = lane + 32 * i < E ? load_factor(__ldg(counts + lane + 32 * i), n, E, top_k) : 0.f;
  for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < tokens; t += (int64_t)gridDim.x * kWarps) {
    float p[kN];
    bool bad = false;
    token_softmax<T, kN>(logits + t * ld, E, lane, p, bad);
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < kN; ++i) dot = fmaf(p[i], f[i], dot);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    T* out = d_logits + t * E;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int e = lane + 32 * i;
      if (e >= E) continue;
      float d = g * p[i] * (f[i] - dot);
      if (accumulate) d += Elem<T>::to_f(out[e]);
      out[e] = to_elem<T>(d);
    }
  }
}

template <typename F>
q4_status by_experts(int E, F&& f) {
  if (E <= 32) return f(std::integral_constant<int, 1>());
  if (E <= 64) return f(std::integral_constant<int, 2>());
  if (E <= 128) return f(std::integral_constant<int, 4>());
  if (E <= 256) return f(std::integral_constant<int, 8>());
  if (E <= 512) return f(std::integral_constant<int, 16>());
  return f(std::integral_constant<int, 32>());
}

int balance_grid(int64_t tokens) {
  return (int)std::max<int64_t>(1, std::min<int64_t>(ceil_div(tokens, 4 * kWarps), 2 * num_sms()));
}

}  // namespace

size_t balance_workspace_bytes(int64_t tokens, int64_t E) {
  return (size_t)balance_grid(tokens) * (size_t)(2 * E + 1) * 4;
}

q4_status launch_balance(const void* logits, int dtype, int64_t tokens, int E, int64_t ld, const int32_t* ids, int top_k,
                         float coeff, float* loss, int32_t* counts, float* mean, void* ws, cudaStream_t stream) {
  const int grid = balance_grid(tokens);
  float* part_p = static_cast<float*>(ws);
  int32_t* part_c = reinterpret_cast<int32_t*>(part_p + (size_t)grid * E);
  const q4_status st = by_dtype(dtype, [&](auto tag) {
    using T = decltype(tag);
    return by_experts(E, [&](auto n) {
      return launch_pdl(balance_kernel<T, decltype(n)::value>, grid, kThreads, 0, stream, static_cast<const T*>(logits), tokens, E,
                        ld, ids, tokens * top_k, part_p, part_c, device_status_ptr());
    });
  });
  if (st != Q4_OK) return st;
  return launch_pdl(balance_finish_kernel, 1, kFinishThreads, 0, stream, static_cast<const float*>(part_p),
                    static_cast<const int32_t*>(part_c), grid, E, top_k, coeff, loss, counts, mean);
}

q4_status launch_balance_backward(const void* logits, int dtype, int64_t tokens, int E, int64_t ld, const int32_t* counts,
                                  int top_k, const float* d_loss, float coeff, bool accumulate, void* d_logits,
                                  cudaStream_t stream) {
  const unsigned grid = (unsigned)std::min<int64_t>(ceil_div(tokens, kWarps), (int64_t)num_sms() * 8);
  return by_dtype(dtype, [&](auto tag) {
    using T = decltype(tag);
    return by_experts(E, [&](auto n) {
      return launch_pdl(balance_backward_kernel<T, decltype(n)::value>, grid, kThreads, 0, stream, static_cast<const T*>(logits),
                        tokens, E, ld, counts, top_k, d_loss, coeff, (int)accumulate, static_cast<T*>(d_logits));
    });
  });
}

}  // namespace q4
