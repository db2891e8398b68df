// Balance loss of the router and its gradient.
//
//   p[t] = softmax(logits[t]) over the experts above -inf;  n: tokens with one
//   counts[e] = slots of expert e,  f[e] = counts[e] E / (n k)
//   P[e] = sum over t of p[t, e] / n,  loss = coeff sum over e of f[e] P[e]
//   d_logits[t, e] = d_loss coeff / n * p[t, e] (f[e] - sum over j of p[t, j] f[j])
// (counts are constants to the gradient).  Softmax and sums are FP32.
//
// A token's logits are held by 1 to 32 lanes, eight neighbouring experts per load
// where rows are aligned (Lanes), else by a warp, lane l the experts l, l + 32, ...;
// its probabilities are added up in registers, token by token.  The blocks' sums
// meet in a fixed order: in distributed shared memory of the same blocks, one
// cluster, where there are few tokens (one_cluster), else in the workspace, from
// where a second kernel adds them (the counts are integers, whose order does not matter).
//
// Not HBM-bound: a token's two reductions and the blocks' join take longer than its
// bytes.  65536 x 256 bf16, top-8 18.8 us with the second kernel, gradient
// 15.6 (4.3 TB/s); 16384 x 64 FP32 7.3 and 3.6; 1000 x 64 6.2 and 2.4 (one cluster:
// launch, one DSMEM exchange, two cluster barriers).
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "elem.cuh"
#include "internal.h"

namespace q4 {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxExperts = 1024;
constexpr int kCluster = 8;
constexpr int kFlight = 8;  // loads of a thread on their way at a time: ids, the blocks' parts
// Loads per lane where there are many logits: fewer lanes share a token and its
// reductions (65536 x 256 bf16, before later steps: 25.9 us with one, 20.6 with two, 19.5
// with four, the gradient 21.0, 17.7 and 31.8; now 18.9 and 15.6 with two); elsewhere
// one (16384 x 64 FP32: 8.2, 8.5 and 11.4).
int loads_of(int64_t tokens, int64_t E) { return tokens * E >= (int64_t)1 << 22 ? 2 : 1; }

// 2^x within 2^-22 relative (0 below 2^-126).
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The lanes that hold a token and their experts: kVec: `lanes` lanes, chunk c of
// lane l the experts 8 (l + lanes c) ...; otherwise a warp, single experts.
template <typename T, bool kVec, int kN>
struct Lanes {
  static constexpr int n = kVec ? 8 * kN : kN;  // experts of a lane
  static constexpr int words = kVec ? kN * 2 * (int)sizeof(T) : kN;
  // -inf, twice in a word of 16-bit elements: what experts behind the last have
  static constexpr uint32_t kMasked = sizeof(T) == 4 ? 0xff800000u : std::is_same<T, __half>::value ? 0xfc00fc00u : 0xff80ff80u;
  int lanes, l, sub, per_warp;
  __device__ __forceinline__ explicit Lanes(int lanes_)
      : lanes(kVec ? lanes_ : 32), l(threadIdx.x & (lanes - 1)), sub((threadIdx.x & 31) / lanes), per_warp(32 / lanes) {}
  __device__ __forceinline__ int expert(int i) const { return kVec ? 8 * (l + lanes * (i / 8)) + i % 8 : l + 32 * i; }
  __device__ __forceinline__ void load(const T* __restrict__ row, int E, bool live, uint32_t (&w)[words]) const {
    if constexpr (kVec) {
      constexpr int per = words / kN / 4;  // 128-bit words of a chunk
#pragma unroll
      for (int c = 0; c < kN; ++c)
#pragma unroll
        for (int i = 0; i < per; ++i) {
          const int e = 8 * (l + lanes * c);
          const uint4 v = live && e < E ? __ldg(reinterpret_cast<const uint4*>(row + e) + i) : make_uint4(kMasked, kMasked, kMasked, kMasked);
          uint32_t* o = w + 4 * (c * per + i);
          o[0] = v.x, o[1] = v.y, o[2] = v.z, o[3] = v.w;
        }
    } else {
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const int e = expert(i);
        if constexpr (sizeof(T) == 2)
          w[i] = live && e < E ? __ldg(reinterpret_cast<const unsigned short*>(row) + e) : kMasked;
        else
          w[i] = live && e < E ? __float_as_uint(__ldg(row + e)) : kMasked;
      }
    }
  }
  static __device__ __forceinline__ float value(const uint32_t (&w)[words], int i) {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    else if constexpr (kVec) {
      const float2 v = unpack2<T>(w[i / 2]);
      return i & 1 ? v.y : v.x;
    } else
      return unpack2<T>(w[i]).x;
  }
  __device__ __forceinline__ float sum(float v) const {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      if (o < lanes) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }
  __device__ __forceinline__ float largest(float v) const {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      if (o < lanes) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
  }
  // exp of a token's logits over the largest, and 1 over their sum (0 and false where
  // every expert is masked).  NaN and +inf mask their expert; they are looked for
  // where the sum shows them.
  __device__ __forceinline__ bool softmax(const uint32_t (&w)[words], float (&p)[n], float& inv, bool& bad) const {
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      p[i] = value(w, i);
      top = fmaxf(top, p[i]);
    }
    top = largest(top);
    float total = exponentials(p, top);
    if (!__all_sync(0xffffffffu, total < INFINITY)) {
      top = -INFINITY;
#pragma unroll
      for (int i = 0; i < n; ++i) {
        p[i] = value(w, i);
        if (!(p[i] < INFINITY)) {
          bad = true;
          p[i] = -INFINITY;
        }
        top = fmaxf(top, p[i]);
      }
      top = largest(top);
      total = exponentials(p, top);
    }
    const bool there = top > -INFINITY;
    inv = there ? __fdividef(1.f, total) : 0.f;
    return there;
  }
  // exp(-d), d = top - x, as 2^(-d log2 e): the difference, the constant (2^-26 off) and
  // the product put the exponent off by 2.25 * 2^-24 of itself, which is that times d
  // relative to the result, and the instruction 2^-22 more: 2^-18 at d = 25.
  __device__ __forceinline__ float exponentials(float (&p)[n], float top) const {
    constexpr float kLog2e = 1.4426950408889634f;
    if (top == -INFINITY) top = 0.f;  // the exponentials are zero then
    float total = 0.f;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      p[i] = exp2_fast((p[i] - top) * kLog2e);
      total += p[i];
    }
    return sum(total);
  }
};

// f[e] from the counts (0 where no token takes part).
__device__ __forceinline__ float load_factor(int32_t count, int32_t n, int E, int top_k) {
  return n > 0 ? (float)count * ((float)E / ((float)n * (float)top_k)) : 0.f;
}

struct FinishArgs {
  int parts, E, top_k;
  float coeff;
  float* part_p;    // [parts, E]; null: the parts are the cluster's, in its shared memory
  int32_t* part_c;  // [parts, E + 1]
  float* loss;
  int32_t* counts;
  float* mean;
};

__device__ __forceinline__ int32_t load_peer(uint32_t addr, uint32_t rank) {
  int32_t v;
  asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(addr, rank)));
  return v;
}

// A cluster's blocks: counts, means and the loss from the parts.  Each block takes
// an eighth of the experts, the threads of an expert every so many-th part; their
// sums meet in a fixed order, and so do the blocks' parts of the loss.
// `scratch`: 2 * blockDim words; own_p, own_c: this block's parts in shared memory.
__device__ __forceinline__ void finish(const FinishArgs& a, uint32_t* scratch, uint32_t own_p, uint32_t own_c) {
  __shared__ int32_t tokens;
  __shared__ float warp_sum[32], block_sum;
  const int threads = blockDim.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rank = (int)cluster_ctarank();
  const int per = (a.E + kCluster - 1) / kCluster, begin = rank * per, end = min(a.E, begin + per);
  int width = 1;  // experts side by side: at most 128
  while (width < per) width *= 2;
  const int groups = threads / width, at = threadIdx.x & (width - 1), group = threadIdx.x / width, e = begin + at;
  float* sp = reinterpret_cast<float*>(scratch);
  int32_t* sc = reinterpret_cast<int32_t*>(scratch + threads);
  auto part_c = [&](int q, int i) {
    return a.part_p ? a.part_c[(int64_t)q * (a.E + 1) + i] : load_peer(own_c + 4 * i, (uint32_t)q);
  };
  if (warp == 0) {
    int32_t n = 0;
    for (int q = lane; q < a.parts; q += 32 * kFlight) {
      int32_t v[kFlight];
#pragma unroll
      for (int u = 0; u < kFlight; ++u) v[u] = q + 32 * u < a.parts ? part_c(q + 32 * u, a.E) : 0;
#pragma unroll
      for (int u = 0; u < kFlight; ++u) n += v[u];
    }
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) tokens = n;
    if (lane == 0 && rank == 0) a.counts[a.E] = n;
  }
  int32_t c = 0;
  float s = 0.f;
  if (e < end) {
    for (int first = group; first < a.parts; first += groups * kFlight) {
      int32_t vc[kFlight];
      float vp[kFlight];
#pragma unroll
      for (int u = 0; u < kFlight; ++u) {
        const int q = first + u * groups;
        const bool there = q < a.parts;
        vc[u] = there ? part_c(q, e) : 0;
        vp[u] = !there ? 0.f : a.part_p ? a.part_p[(int64_t)q * a.E + e] : __int_as_float(load_peer(own_p + 4 * e, (uint32_t)q));
      }
#pragma unroll
      for (int u = 0; u < kFlight; ++u) c += vc[u], s += vp[u];
    }
  }
  sp[threadIdx.x] = s;
  sc[threadIdx.x] = c;
  // the groups meet in pairs
  for (int g = groups / 2; g > 0; g /= 2) {
    __syncthreads();
    if (group < g) {
      sp[threadIdx.x] += sp[threadIdx.x + g * width];
      sc[threadIdx.x] += sc[threadIdx.x + g * width];
    }
  }
  __syncthreads();
  float part = 0.f;
  if (group == 0 && e < end) {
    const int32_t n = tokens;
    const float m = n > 0 ? __fdiv_rn(sp[threadIdx.x], (float)n) : 0.f;
    a.counts[e] = sc[threadIdx.x];
    a.mean[e] = m;
    part = load_factor(sc[threadIdx.x], n, a.E, a.top_k) * m;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
  if (lane == 0) warp_sum[warp] = part;
  __syncthreads();
  if (threadIdx.x == 0) {
    float sum = 0.f;
    for (int w = 0; w < (width + 31) / 32; ++w) sum += warp_sum[w];  // group 0's warps
    block_sum = sum;
  }
  cluster_barrier_sync();  // every block's part of the loss is there
  if (rank == 0 && threadIdx.x == 0) {
    float sum = 0.f;
    for (int b = 0; b < kCluster; ++b)
      sum += __int_as_float(load_peer(smem_u32(&block_sum), (uint32_t)b));
    *a.loss = a.coeff * sum;
  }
  cluster_barrier_sync();  // no block leaves before its part was read
}

template <typename T, bool kVec, int kN>
__global__ void __launch_bounds__(kThreads)
    balance_kernel(const T* __restrict__ logits, int64_t tokens, int64_t ld, const int32_t* __restrict__ ids, int lanes,
                   const FinishArgs f, int* status) {
  pdl_wait();
  using L = Lanes<T, kVec, kN>;
  // the warps' sums one after another where all do not fit: 16 warps x 1024 experts
  constexpr int kSumWarps = 8;
  __shared__ float sum[kSumWarps * kMaxExperts];
  __shared__ float total[kMaxExperts];
  __shared__ int32_t count[kMaxExperts + 1];
  const L lay(lanes);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = f.E;
  for (int e = threadIdx.x; e <= E; e += kThreads) count[e] = 0;
  __syncthreads();
  // the next token's logits are on their way while this one's are worked on
  const int64_t step = (int64_t)gridDim.x * kWarps * lay.per_warp;
  int64_t t = ((int64_t)blockIdx.x * kWarps + warp) * lay.per_warp + lay.sub;
  uint32_t w[L::words];
  lay.load(logits + t * ld, E, t < tokens, w);
  const int64_t slots = tokens * f.top_k, stride = (int64_t)gridDim.x * kThreads;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < slots; i += kFlight * stride) {
    int id[kFlight];
#pragma unroll
    for (int u = 0; u < kFlight; ++u) id[u] = i + u * stride < slots ? __ldg(ids + i + u * stride) : -1;
#pragma unroll
    for (int u = 0; u < kFlight; ++u)
      if (id[u] >= 0 && id[u] < E) atomicAdd(&count[id[u]], 1);
  }
  float acc[L::n];
#pragma unroll
  for (int i = 0; i < L::n; ++i) acc[i] = 0.f;
  int there = 0;
  bool bad = false;
  for (int64_t first = t - lay.sub; first < tokens; first += step, t += step) {
    uint32_t next[L::words];
    lay.load(logits + (t + step) * ld, E, t + step < tokens, next);
    float p[L::n], inv;
    there += lay.softmax(w, p, inv, bad) && lay.l == 0;
#pragma unroll
    for (int i = 0; i < L::n; ++i) acc[i] = fmaf(p[i], inv, acc[i]);
#pragma unroll
    for (int i = 0; i < L::words; ++i) w[i] = next[i];
  }
  if (bad) latch_status(status, Q4_ERR_NONFINITE);
  there = __reduce_add_sync(0xffffffffu, there);
  if (lane == 0) atomicAdd(&count[E], there);
  // lanes of several tokens hold the same experts
  for (int o = lay.lanes; o < 32; o <<= 1) {
#pragma unroll
    for (int i = 0; i < L::n; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
  }
#pragma unroll
  for (int turn = 0; turn < kWarps / kSumWarps; ++turn) {
    if (warp / kSumWarps == turn && lay.sub == 0) {
      float* to = sum + warp % kSumWarps * kMaxExperts;
#pragma unroll
      for (int i = 0; i < L::n; ++i) {
        const int e = lay.expert(i);
        if (e < E) to[e] = turn ? to[e] + acc[i] : acc[i];
      }
    }
    __syncthreads();
  }
  for (int e = threadIdx.x; e <= E; e += kThreads) {
    float s = 0.f;
    if (e < E) {
#pragma unroll
      for (int i = 0; i < kSumWarps; ++i) s += sum[i * kMaxExperts + e];
    }
    if (f.part_p) {
      f.part_c[(int64_t)blockIdx.x * (E + 1) + e] = count[e];
      if (e < E) f.part_p[(int64_t)blockIdx.x * E + e] = s;
    } else if (e < E) {
      total[e] = s;
    }
  }
  if (f.part_p) return;
  cluster_barrier_sync();  // the cluster's parts are there
  finish(f, reinterpret_cast<uint32_t*>(sum), smem_u32(total), smem_u32(count));
}

// Threads of its blocks: more where they have parts of many experts to add up (16384 x
// 64 FP32: 7.3 us with 512 threads, 7.9 with 1024; 8192 x 1024 bf16 19.8 and 18.4;
// starting it early, to wait beside the first kernel's blocks, changed nothing).
constexpr int kFinishThreads = 1024;
int finish_threads(int E) { return E <= 256 ? kFinishThreads / 2 : kFinishThreads; }
__global__ void __launch_bounds__(kFinishThreads) balance_finish_kernel(const FinishArgs f) {
  pdl_wait();
  __shared__ uint32_t scratch[2 * kFinishThreads];
  finish(f, scratch, 0, 0);
}

// Blocks of the gradient per SM, all resident: a second wave repeats the counts' way
// from memory (six blocks for all: 65536 x 256 bf16 17.7 us instead of 15.7, 8192 x
// 1024 25.9 instead of 18.9, 32768 x 64 5.8 instead of 4.6).
constexpr int gradient_blocks(bool vec, int n) { return vec ? (n == 1 ? 4 : n == 2 ? 3 : 2) : n <= 8 ? 4 : 2; }

template <typename T, bool kVec, int kN>
__global__ void __launch_bounds__(256, gradient_blocks(kVec, kN))
    balance_backward_kernel(const T* __restrict__ logits, int64_t tokens, int E, int64_t ld, const int32_t* __restrict__ counts,
                            int lanes, int top_k, const float* __restrict__ d_loss, float coeff, int accumulate,
                            T* __restrict__ d_logits) {
  pdl_wait();
  using L = Lanes<T, kVec, kN>;
  const L lay(lanes);
  const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int64_t step = (int64_t)gridDim.x * warps * lay.per_warp;
  int64_t t = ((int64_t)blockIdx.x * warps + warp) * lay.per_warp + lay.sub;
  uint32_t w[L::words];
  lay.load(logits + t * ld, E, t < tokens, w);
  const int32_t n = __ldg(counts + E);
  const float g = n > 0 ? __ldg(d_loss) * __fdiv_rn(coeff, (float)n) : 0.f;
  float f[L::n];
#pragma unroll
  for (int i = 0; i < L::n; ++i) f[i] = lay.expert(i) < E ? load_factor(__ldg(counts + lay.expert(i)), n, E, top_k) : 0.f;
  for (int64_t first = t - lay.sub; first < tokens; first += step, t += step) {
    uint32_t next[L::words];
    lay.load(logits + (t + step) * ld, E, t + step < tokens, next);
    const bool live = t < tokens;
    float p[L::n], inv;
    bool bad = false;
    lay.softmax(w, p, inv, bad);
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < L::n; ++i) dot = fmaf(p[i], f[i], dot);
    dot = lay.sum(dot) * inv;
    inv *= g;
    T* out = d_logits + t * E;
#pragma unroll
    for (int i = 0; i < L::n; ++i) p[i] = inv * p[i] * (f[i] - dot);
    if constexpr (kVec) {
#pragma unroll
      for (int c = 0; c < kN; ++c) {
        const int e = 8 * (lay.l + lay.lanes * c);
        if (!live || e >= E) continue;
        uint4* to = reinterpret_cast<uint4*>(out + e);
        float* d = p + 8 * c;
        if (accumulate) {
#pragma unroll
          for (int i = 0; i < 8; ++i) d[i] += Elem<T>::to_f(out[e + i]);
        }
        if constexpr (sizeof(T) == 4) {
          to[0] = make_uint4(__float_as_uint(d[0]), __float_as_uint(d[1]), __float_as_uint(d[2]), __float_as_uint(d[3]));
          to[1] = make_uint4(__float_as_uint(d[4]), __float_as_uint(d[5]), __float_as_uint(d[6]), __float_as_uint(d[7]));
        } else {
          to[0] = make_uint4(pack2<T>(d[0], d[1]), pack2<T>(d[2], d[3]), pack2<T>(d[4], d[5]), pack2<T>(d[6], d[7]));
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < L::n; ++i) {
        const int e = lay.expert(i);
        if (!live || e >= E) continue;
        if (accumulate) p[i] += Elem<T>::to_f(out[e]);
        out[e] = to_elem<T>(p[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < L::words; ++i) w[i] = next[i];
  }
}

// The kernels' forms: eight experts per load (kVec) with 1, 2 or 4 loads per lane, at
// least `loads` where there are as many, or single experts, 2 to 32 per lane.
template <typename F>
q4_status by_experts(bool vec, int E, int loads, F&& f) {
  if (vec) {
    if (E <= 256 && (loads == 1 || E <= 8)) return f(std::true_type(), std::integral_constant<int, 1>());
    if (E <= 512 && (loads <= 2 || E <= 16)) return f(std::true_type(), std::integral_constant<int, 2>());
    return f(std::true_type(), std::integral_constant<int, 4>());
  }
  if (E <= 64) return f(std::false_type(), std::integral_constant<int, 2>());
  if (E <= 256) return f(std::false_type(), std::integral_constant<int, 8>());
  return f(std::false_type(), std::integral_constant<int, 32>());
}
// Lanes of a token with `loads` loads each.
int lanes_of(bool vec, int E, int loads) {
  int lanes = 1;
  while (lanes < 32 && 8 * loads * lanes < E) lanes *= 2;
  return vec ? lanes : 32;
}

// Blocks: a cluster that finishes by itself where a warp has few tokens, four turns of
// 256 experts or (more of them, or widths that eight do not divide) of a token, else
// one per SM and a second launch.  FP32, cluster and grid: 1000 x 64 6.1 and 7.5 us,
// 2000 x 64 7.2 and 7.5, 8192 x 64 12.0 and 7.6, 256 x 256 6.3 and 8.7, 1000 x 256 9.2
// and 8.7, 512 x 1024 14.3 and 16.9, 500 x 60 5.8 and 7.0, 2000 x 60 9.2 and 7.0.
bool one_cluster(int64_t tokens, int64_t E) {
  return tokens * (E % 8 ? 256 : std::min<int64_t>(E, 256)) <= (int64_t)kCluster * kWarps * 4 * 256;
}
int balance_grid(int64_t tokens, int64_t E) { return one_cluster(tokens, E) ? kCluster : num_sms(); }

// Programmatic dependent launch, and clusters of kCluster blocks.
void cluster_attributes(cudaLaunchAttribute (&attr)[2]) {
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kCluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
}

}  // namespace

size_t balance_workspace_bytes(int64_t tokens, int64_t E) {
  return one_cluster(tokens, E) ? 0 : (size_t)balance_grid(tokens, E) * (size_t)(2 * E + 1) * 4;
}

q4_status launch_balance(const void* logits, int dtype, int64_t tokens, int E, int64_t ld, const int32_t* ids, int top_k,
                         float coeff, float* loss, int32_t* counts, float* mean, void* ws, cudaStream_t stream) {
  const int grid = balance_grid(tokens, E);
  const bool all = one_cluster(tokens, E);
  FinishArgs f = {grid, E, top_k, coeff, all ? nullptr : static_cast<float*>(ws), nullptr, loss, counts, mean};
  if (!all) f.part_c = reinterpret_cast<int32_t*>(f.part_p + (size_t)grid * E);
  const bool vec = E % 8 == 0 && ld * (dtype == Q4_F32 ? 4 : 2) % 16 == 0 && mult(logits, 16);
  const q4_status st = by_dtype(dtype, [&](auto tag) {
    using T = decltype(tag);
    return by_experts(vec, E, all ? 1 : loads_of(tokens, E), [&](auto v, auto n) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3((unsigned)grid, 1, 1);
      cfg.blockDim = dim3(kThreads, 1, 1);
      cfg.stream = stream;
      cudaLaunchAttribute attr[2];
      cluster_attributes(attr);
      cfg.attrs = attr;
      cfg.numAttrs = all ? 2 : 1;
      return cudaLaunchKernelEx(&cfg, balance_kernel<T, decltype(v)::value, decltype(n)::value>, static_cast<const T*>(logits),
                                tokens, ld, ids, lanes_of(vec, E, decltype(n)::value), f, device_status_ptr()) == cudaSuccess
                 ? Q4_OK
                 : Q4_ERR_CUDA;
    });
  });
  if (st != Q4_OK || all) return st;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kCluster, 1, 1);
  cfg.blockDim = dim3((unsigned)finish_threads(E), 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  cluster_attributes(attr);
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  Q4_CUDA_TRY(cudaLaunchKernelEx(&cfg, balance_finish_kernel, f));
  return Q4_OK;
}

q4_status launch_balance_backward(const void* logits, int dtype, int64_t tokens, int E, int64_t ld, const int32_t* counts,
                                  int top_k, const float* d_loss, float coeff, bool accumulate, void* d_logits,
                                  cudaStream_t stream) {
  const bool vec = E % 8 == 0 && ld * (dtype == Q4_F32 ? 4 : 2) % 16 == 0 && mult(logits, 16) && mult(d_logits, 16);
  return by_dtype(dtype, [&](auto tag) {
    using T = decltype(tag);
    return by_experts(vec, E, loads_of(tokens, E), [&](auto v, auto n) {
      const int lanes = lanes_of(vec, E, decltype(n)::value), per_block = 8 * (32 / lanes);  // tokens at a time
      const unsigned grid = (unsigned)std::min<int64_t>(ceil_div(tokens, per_block), (int64_t)num_sms() * gradient_blocks(vec, decltype(n)::value));
      return launch_pdl(balance_backward_kernel<T, decltype(v)::value, decltype(n)::value>, grid, 256, 0, stream,
                        static_cast<const T*>(logits), tokens, E, ld, counts, lanes, top_k, d_loss, coeff, (int)accumulate,
                        static_cast<T*>(d_logits));
    });
  });
}

}  // namespace q4
