// Routing of tokens to experts around the grouped products: top-k with softmax
// weights, tokens sorted by expert, rows brought into expert order and back,
// and the gradients of these.
//
// With l the logits of a token, V its experts with l > -inf and C the top_k
// of V by logit (ties to the lower index):
//   weights   w_j = exp(l_j - m) / sum_{i in C or V} exp(l_i - m),  m = max l
//   gradient  over C: dl_j = w_j (dw_j - sum_i dw_i w_i), zero elsewhere;
//             over V: dl_e = p_e (g_e - sum_i dw_i p_i), g_e = dw_j for the
//             chosen expert of slot j and 0 otherwise.
// A slot (t, j) has a row in expert order; slot_row holds that row, or ~row
// for a slot that was dropped (its row lies behind every expert's rows):
//   dispatch  rows[row(t, j)] = x[t]                (zero for a dropped slot)
//   combine   out[t] = sum_j w_tj rows[row(t, j)]   (dropped slots left out)
//   gradient  d_rows[row(t, j)] = w_tj d_out[t],  dw_tj = <d_out[t], rows[row(t, j)]>
#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace q4 {
namespace {

constexpr int kWarp = 32;
constexpr unsigned kFull = 0xffffffffu;

template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }

// ------------------------------------------------------------------ routing
// One element as a float.  16-bit elements come through a whole register: loads
// into half a register wait for one another.
template <typename T>
__device__ __forceinline__ float load_float(const T* p) {
  if constexpr (sizeof(T) == 4) {
    return __ldg(p);
  } else {
    const unsigned short b = __ldg(reinterpret_cast<const unsigned short*>(p));
    return Elem<T>::to_f(*reinterpret_cast<const T*>(&b));
  }
}

// The weights' exponential: within 2 + 1.2 |x| ulp, x = l - m <= 0, so the
// relative error grows only where the weight itself is small.
__device__ __forceinline__ float weight_exp(float x) { return __expf(x); }

// The logit of an FP32 key (Keys below).
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// A lane's experts, lane + 32 i, by an unsigned key that orders logits as
// numbers do (-0 equal to +0); 0 for a masked expert: -inf, or a NaN or +inf,
// which are latched as errors.  The key of a 16-bit logit fits in 16 bits
// beside its expert (0xffff - e: the lower index wins a tie), which makes a
// round one maximum over the warp; FP32 keys need the index found after it.
// The keys stand in groups with their maxima kept, so that a round looks at
// the maxima and at one group, the same for the whole warp, instead of at all
// keys (16384 x 1024, top-8: 72 -> 47 us in FP32, 49 -> 42 us in bf16; with all
// loads ahead of the first key 29 and 26).
template <typename T, int NV>
struct Keys {
  static constexpr bool kPacked = sizeof(T) == 2;
  static constexpr int kGroup = NV <= 4 ? NV : NV <= 8 ? 4 : 8, kGroups = NV / kGroup;
  uint32_t key[NV], top[kGroups];

  __device__ __forceinline__ void load(const T* row, int E, int lane, bool& bad) {
    // 16-bit elements by way of whole registers, so that no load waits for another
    constexpr uint32_t kInf = kPacked ? (std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u) : 0x7f800000u;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = lane + 32 * i;
      if constexpr (kPacked)
        key[i] = e < E ? (uint32_t)__ldg(reinterpret_cast<const unsigned short*>(row) + e) : 0x8000u | kInf;
      else
        key[i] = e < E ? __float_as_uint(__ldg(row + e)) : 0x80000000u | kInf;  // -inf
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      constexpr uint32_t kSign = kPacked ? 0x8000u : 0x80000000u;
      const uint32_t b = key[i];
      // NaN and +inf are errors; they and -inf are masked
      const bool masked = (b & ~kSign) >= kInf;
      bad |= masked && b != (kSign | kInf);
      // positive numbers above negative ones, the order of those turned; -0 as +0
      const uint32_t k = b & kSign && b != kSign ? ~b : b | kSign;
      if constexpr (kPacked)
        key[i] = masked ? 0u : k << 16 | (0xffffu - (lane + 32 * i));
      else
        key[i] = masked ? 0u : k;
    }
#pragma unroll
    for (int g = 0; g < kGroups; ++g) top_of(g);
  }
  __device__ __forceinline__ void top_of(int g) {
    top[g] = key[g * kGroup];
#pragma unroll
    for (int i = 1; i < kGroup; ++i) top[g] = max(top[g], key[g * kGroup + i]);
  }
  // The warp's largest key (0: none left).
  __device__ __forceinline__ uint32_t largest() const {
    uint32_t best = top[0];
#pragma unroll
    for (int g = 1; g < kGroups; ++g) best = max(best, top[g]);
    return __reduce_max_sync(kFull, best);
  }
  __device__ static __forceinline__ float value(uint32_t k) {
    if constexpr (kPacked) {
      const uint16_t b = (uint16_t)(k & 0x80000000u ? k >> 16 & 0x7fffu : ~(k >> 16));
      return Elem<T>::to_f(*reinterpret_cast<const T*>(&b));
    } else {
      return key_value(k);
    }
  }
  // Takes the largest key m out; its expert, the lowest one if several have it.
  __device__ __forceinline__ int pop(uint32_t m, int lane) {
    uint32_t in = kGroups;  // the group it is in
    if constexpr (kPacked) {
      in = (0xffffu - (m & 0xffffu)) / 32 / kGroup;
    } else {
#pragma unroll
      for (int g = kGroups - 1; g >= 0; --g)
        if (top[g] == m) in = g;
      if constexpr (kGroups > 1) in = __reduce_min_sync(kFull, in);
      else in = 0;
    }
    uint32_t at = kPacked ? 0xffffu - (m & 0xffffu) : 0xffffffffu;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      if (in != (uint32_t)g) continue;  // the same for the whole warp
      if constexpr (!kPacked) {
#pragma unroll
        for (int i = kGroup - 1; i >= 0; --i)
          if (key[g * kGroup + i] == m) at = (uint32_t)(lane + 32 * (g * kGroup + i));
        at = __reduce_min_sync(kFull, at);
      }
#pragma unroll
      for (int i = 0; i < kGroup; ++i)
        if (at == (uint32_t)(lane + 32 * (g * kGroup + i))) key[g * kGroup + i] = 0u;
      top_of(g);
    }
    return (int)at;
  }
};

constexpr int kRouteWarps = 4;

// One warp per token.  Bound by the integer pipe in the rounds (69% of the issue
// slots while the SMs run, 4.7 warps ready per cycle, the others waiting for that
// pipe rather than for memory): 16384 x 256 bf16, top-8 and softmax over all, takes
// 12.1 us (its gradient 6.2, waiting for its loads), where reading the 8 MB takes 1.2
// at the copy rate.
template <typename T, int NV>
__global__ void __launch_bounds__(kRouteWarps * kWarp)
    route_kernel(const T* __restrict__ logits, int64_t tokens, int E, int64_t ld, int top_k, int over_all,
                 int32_t* __restrict__ ids, float* __restrict__ weights, int* status) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
  if (t >= tokens) return;
  Keys<T, NV> keys;
  bool bad = false;
  keys.load(logits + t * ld, E, lane, bad);
  if (__any_sync(kFull, bad) && lane == 0) latch_status(status, Q4_ERR_NONFINITE);
  uint32_t m = keys.largest();
  const float top = m ? Keys<T, NV>::value(m) : 0.f;
  float sum = 0.f, mine = 0.f;
  if (over_all) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (keys.key[i]) sum += weight_exp(Keys<T, NV>::value(keys.key[i]) - top);
  }
  int my_id = -1;
  uint32_t my_key = 0;
  for (int j = 0; j < top_k && m; ++j) {
    const int id = keys.pop(m, lane);
    if (lane == j) my_id = id, my_key = m;
    m = keys.largest();
  }
  if (my_key) mine = weight_exp(Keys<T, NV>::value(my_key) - top);
  if (!over_all) sum = mine;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  if (lane < top_k) {
    ids[t * top_k + lane] = my_id;
    weights[t * top_k + lane] = my_id < 0 ? 0.f : mine / sum;
  }
}

// The gradient; one warp per token, lane j also holds slot j.  The maximum
// and sum are taken again from the logits, which have to be read anyway.
// -p_e sum_i dw_i p_i (or 0) goes to every expert, then the slots' lanes
// replace the chosen ones' by w_j (dw_j - sum_i dw_i w_i).
template <typename T, int NV>
__global__ void __launch_bounds__(kRouteWarps * kWarp)
    route_backward_kernel(const T* __restrict__ logits, int64_t tokens, int E, int64_t ld, int top_k,
                          int over_all, const int32_t* __restrict__ ids,
                          const float* __restrict__ d_weights, T* __restrict__ d_logits) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
  if (t >= tokens) return;
  const T* row = logits + t * ld;
  int id = lane < top_k ? ids[t * top_k + lane] : -1;
  if ((unsigned)id >= (unsigned)E) id = -1;
  const float mine = id >= 0 ? load_float(row + id) : 0.f;
  const bool live = id >= 0 && !nonfinite(mine);
  const float dw = live ? d_weights[t * top_k + lane] : 0.f;
  const float kLow = -__int_as_float(0x7f800000);
  float p[NV];  // the logits, -inf where masked
  float top = live ? mine : kLow;
  if (over_all) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = lane + 32 * i;
      p[i] = e < E ? load_float(row + e) : kLow;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (nonfinite(p[i])) p[i] = kLow;
      top = fmaxf(top, p[i]);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
  if (top == kLow) top = 0.f;  // no expert at all
  const float w = live ? weight_exp(mine - top) : 0.f;
  float sum = over_all ? 0.f : w, dot = w * dw;
  if (over_all) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      p[i] = weight_exp(p[i] - top);
      sum += p[i];
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(kFull, sum, o);
    dot += __shfl_xor_sync(kFull, dot, o);
  }
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  dot *= inv;
  T* out = d_logits + t * E;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane + 32 * i;
    if (e < E) out[e] = from_f<T>(over_all ? -p[i] * inv * dot : 0.f);
  }
  __syncwarp();  // orders the slots' stores behind these
  if (live) out[id] = from_f<T>(w * inv * (dw - dot));
}

// ------------------------------------------------------------------ sort
// A stable counting sort of the S = T top_k slots by expert (bucket E holds
// the dropped ones): chunk histograms, one scan per expert over the chunks,
// then every chunk places its slots.  524288 slots of 256 experts take 17 us, of
// which little is traffic (6 MB): three kernels that depend on one another
// (started early, to wait beside the one before, 26 us).
constexpr int kSortThreads = 256, kSortWarps = kSortThreads / 32;
constexpr int kSortChunk = 1024, kSortPerWarp = kSortChunk / kSortWarps;

__device__ __forceinline__ int sort_bucket(const int32_t* __restrict__ ids, int64_t i, int E) {
  const int e = __ldg(ids + i);
  return (unsigned)e < (unsigned)E ? e : E;
}

__global__ void __launch_bounds__(kSortThreads)
    sort_count_kernel(const int32_t* __restrict__ ids, int64_t S, int E, int chunks, int32_t* __restrict__ hist) {
  pdl_wait();
  extern __shared__ int32_t cnt[];
  for (int e = threadIdx.x; e <= E; e += kSortThreads) cnt[e] = 0;
  __syncthreads();
  const int64_t base = (int64_t)blockIdx.x * kSortChunk;
  for (int i = threadIdx.x; i < kSortChunk && base + i < S; i += kSortThreads)
    atomicAdd(cnt + sort_bucket(ids, base + i, E), 1);
  __syncthreads();
  for (int e = threadIdx.x; e <= E; e += kSortThreads) hist[(int64_t)e * chunks + blockIdx.x] = cnt[e];
}

// Block e: exclusive prefix of expert e's chunk counts, and their total.
__global__ void __launch_bounds__(kSortThreads)
    sort_scan_kernel(int chunks, int32_t* __restrict__ hist, int32_t* __restrict__ total) {
  pdl_wait();
  __shared__ int32_t warp_sum[kSortWarps];
  int32_t* h = hist + (int64_t)blockIdx.x * chunks;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int carry = 0;
  for (int c0 = 0; c0 < chunks; c0 += kSortThreads) {
    const int c = c0 + threadIdx.x;
    const int v = c < chunks ? h[c] : 0;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    int before = carry, all = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
      if (w < warp) before += warp_sum[w];
      all += warp_sum[w];
    }
    if (c < chunks) h[c] = before + x - v;
    carry += all;
    __syncthreads();
  }
  if (threadIdx.x == 0) total[blockIdx.x] = carry;
}

__global__ void __launch_bounds__(kSortThreads)
    sort_place_kernel(const int32_t* __restrict__ ids, int64_t S, int E, int top_k, int chunks,
                      const int32_t* __restrict__ hist, const int32_t* __restrict__ total,
                      int32_t* __restrict__ offsets, int32_t* __restrict__ row_token,
                      int32_t* __restrict__ slot_row) {
  pdl_wait();
  extern __shared__ int32_t cnt[];  // [kSortWarps][E + 1], then [E + 1] first rows of the experts
  __shared__ int32_t warp_sum[kSortWarps];
  const int nb = E + 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int32_t* first = cnt + kSortWarps * nb;
  for (int i = threadIdx.x; i < kSortWarps * nb; i += kSortThreads) cnt[i] = 0;
  // exclusive prefix of the experts' totals
  int carry = 0;
  for (int e0 = 0; e0 < nb; e0 += kSortThreads) {
    const int e = e0 + threadIdx.x;
    const int v = e < nb ? total[e] : 0;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    int before = carry, all = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
      if (w < warp) before += warp_sum[w];
      all += warp_sum[w];
    }
    if (e < nb) {
      first[e] = before + x - v;
      if (blockIdx.x == 0) offsets[e] = before + x - v;
    }
    carry += all;
    __syncthreads();
  }
  const int64_t base = (int64_t)blockIdx.x * kSortChunk + warp * kSortPerWarp;
  int32_t* mine = cnt + warp * nb;
  for (int i = 0; i < kSortPerWarp; i += 32) {
    const int64_t s = base + i + lane;
    const int b = s < S ? sort_bucket(ids, s, E) : -1;
    const unsigned peers = __match_any_sync(kFull, b);
    if (b >= 0 && lane == __ffs(peers) - 1) mine[b] += __popc(peers);
    __syncwarp();
  }
  __syncthreads();
  for (int e = threadIdx.x; e < nb; e += kSortThreads) {
    int at = first[e] + hist[(int64_t)e * chunks + blockIdx.x];
    for (int w = 0; w < kSortWarps; ++w) {
      const int c = cnt[w * nb + e];
      cnt[w * nb + e] = at;
      at += c;
    }
  }
  __syncthreads();
  for (int i = 0; i < kSortPerWarp; i += 32) {
    const int64_t s = base + i + lane;
    const int b = s < S ? sort_bucket(ids, s, E) : -1;
    const unsigned peers = __match_any_sync(kFull, b);
    int row = 0;
    if (b >= 0) row = mine[b] + __popc(peers & ((1u << lane) - 1u));
    __syncwarp();
    if (b >= 0 && lane == __ffs(peers) - 1) mine[b] += __popc(peers);
    __syncwarp();
    if (b >= 0) {
      row_token[row] = (int32_t)(s / top_k);
      slot_row[s] = b < E ? row : ~row;
    }
  }
}

// The whole sort in one launch of one cluster: every block takes a contiguous
// share of the slots, every warp of it a contiguous part of that.  The blocks'
// histograms meet in distributed shared memory, and each block computes the
// first row of its own slots of every expert from them.
constexpr int kClusterThreads = 512, kClusterWarps = kClusterThreads / 32, kMaxCluster = 8;

__device__ __forceinline__ int32_t load_peer(uint32_t addr, uint32_t rank) {
  int32_t v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(addr, rank)) : "memory");
  return v;
}

// smem: [warps][E + 1] counts of the warps, then [E + 1] of the block.
__global__ void __launch_bounds__(kClusterThreads)
    sort_cluster_kernel(const int32_t* __restrict__ ids, int S, int E, int top_k, int per_warp,
                        int32_t* __restrict__ offsets, int32_t* __restrict__ row_token,
                        int32_t* __restrict__ slot_row) {
  pdl_wait();
  extern __shared__ int32_t cnt[];
  __shared__ int32_t warp_sum[kClusterWarps];
  const int nb = E + 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int rank = blockIdx.x, blocks = gridDim.x;
  int32_t* own = cnt + warps * nb;
  for (int i = threadIdx.x; i < warps * nb; i += blockDim.x) cnt[i] = 0;
  __syncthreads();
  const int base = (rank * warps + warp) * per_warp;
  const int end = min(base + per_warp, S);
  int32_t* mine = cnt + warp * nb;
  for (int s0 = base; s0 < end; s0 += 32) {
    const int b = s0 + lane < end ? sort_bucket(ids, s0 + lane, E) : -1;
    const unsigned peers = __match_any_sync(kFull, b);
    if (b >= 0 && lane == __ffs(peers) - 1) mine[b] += __popc(peers);
    __syncwarp();
  }
  __syncthreads();
  for (int e = threadIdx.x; e < nb; e += blockDim.x) {
    int sum = 0;
#pragma unroll 8
    for (int w = 0; w < warps; ++w) sum += cnt[w * nb + e];
    own[e] = sum;
  }
  if (blocks > 1)
    cluster_barrier_sync();  // every block's histogram is there
  else
    __syncthreads();
  // first row of expert e: the totals of the experts before it; of this
  // block's slots of e: plus the counts of the blocks before this one
  int carry = 0;
  for (int e0 = 0; e0 < nb; e0 += blockDim.x) {
    const int e = e0 + threadIdx.x;
    int total = 0, before = 0;
    if (e < nb)
      for (int r = 0; r < blocks; ++r) {
        const int c = r == rank ? own[e] : load_peer(smem_u32(own + e), r);
        total += c;
        if (r < rank) before += c;
      }
    int x = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    int prefix = carry, all = 0;
    for (int w = 0; w < warps; ++w) {
      if (w < warp) prefix += warp_sum[w];
      all += warp_sum[w];
    }
    if (e < nb) {
      const int first = prefix + x - total;
      if (rank == 0) offsets[e] = first;
      int at = first + before;
      for (int w0 = 0; w0 < warps; w0 += 8) {  // eight loads in flight
        int c[8];
#pragma unroll
        for (int w = 0; w < 8; ++w) c[w] = w0 + w < warps ? cnt[(w0 + w) * nb + e] : 0;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
          if (w0 + w < warps) cnt[(w0 + w) * nb + e] = at;
          at += c[w];
        }
      }
    }
    carry += all;
    __syncthreads();
  }
  for (int s0 = base; s0 < end; s0 += 32) {
    const int s = s0 + lane;
    const int b = s < end ? sort_bucket(ids, s, E) : -1;
    const unsigned peers = __match_any_sync(kFull, b);
    int row = 0;
    if (b >= 0) row = mine[b] + __popc(peers & ((1u << lane) - 1u));
    __syncwarp();
    if (b >= 0 && lane == __ffs(peers) - 1) mine[b] += __popc(peers);
    __syncwarp();
    if (b >= 0) {
      row_token[row] = s / top_k;
      slot_row[s] = b < E ? row : ~row;
    }
  }
  if (blocks > 1) cluster_barrier_sync();  // no block leaves while a peer reads its histogram
}

// ------------------------------------------------------------------ dispatch / combine
// A row is cut into units of kBytes: 16 where the width, pitches and addresses
// allow it, else 4 (two 16-bit elements), else single elements.  A unit stays
// the words that it was loaded as: an array of 16-bit elements takes a register
// for each of them (107 registers instead of 64 in combine_backward_kernel, and
// half its rate), and loads into half a register wait for one another (single
// bf16 elements, 2048 x 4097, top-8: combine 49 us instead of 85, its gradient
// 89 instead of 286; in units of 4 bytes at 4098: 36 and 60).
template <typename T>
__device__ __forceinline__ float2 unpack(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 unpack<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <typename T>
__device__ __forceinline__ uint32_t pack(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack<__half>(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

template <typename T, int kBytes>
struct Unit {
  static constexpr int n = kBytes / (int)sizeof(T), words = kBytes < 4 ? 1 : kBytes / 4;
  static constexpr bool packed = sizeof(T) == 2 && kBytes >= 4;
  uint32_t w[words];  // a single 16-bit element: in the low half, the high one zero

  // kConst: of memory that this launch does not write.
  template <bool kConst = true>
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kBytes == 16) {
      const uint4 v = word<kConst, uint4>(p);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else if constexpr (kBytes == 4) {
      w[0] = word<kConst, uint32_t>(p);
    } else {
      w[0] = word<kConst, unsigned short>(p);
    }
  }
  template <bool kConst, typename W>
  static __device__ __forceinline__ W word(const T* p) {
    if constexpr (kConst)
      return __ldg(reinterpret_cast<const W*>(p));
    else
      return *reinterpret_cast<const W*>(p);
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (kBytes == 16)
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (kBytes == 4)
      *reinterpret_cast<uint32_t*>(p) = w[0];
    else
      *reinterpret_cast<unsigned short*>(p) = (unsigned short)w[0];
  }
  __device__ __forceinline__ void floats(float (&f)[n]) const {
    if constexpr (packed) {
#pragma unroll
      for (int i = 0; i < words; ++i) {
        const float2 v = unpack<T>(w[i]);
        f[2 * i] = v.x, f[2 * i + 1] = v.y;
      }
    } else if constexpr (sizeof(T) == 2) {
      f[0] = unpack<T>(w[0]).x;
    } else {
#pragma unroll
      for (int i = 0; i < n; ++i) f[i] = __uint_as_float(w[i]);
    }
  }
  __device__ __forceinline__ void round(const float (&f)[n]) {
    if constexpr (packed) {
#pragma unroll
      for (int i = 0; i < words; ++i) w[i] = pack<T>(f[2 * i], f[2 * i + 1]);
    } else if constexpr (sizeof(T) == 2) {
      w[0] = pack<T>(f[0], 0.f);
    } else {
#pragma unroll
      for (int i = 0; i < n; ++i) w[i] = __float_as_uint(f[i]);
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < words; ++i) w[i] = 0u;
  }
};

// blockIdx.x: token; the units of its row are spread over blockIdx.y.  Bound by
// the writes: 4096 x 7168 bf16, top-8, 83 us (6.4 TB/s; a warp per slot the same).
template <typename T, int kBytes>
__global__ void __launch_bounds__(256)
    dispatch_kernel(const T* __restrict__ x, int64_t ldx, int64_t H, const int32_t* __restrict__ slot_row,
                    int top_k, uint32_t S, T* __restrict__ rows) {
  pdl_wait();
  constexpr int n = Unit<T, kBytes>::n;
  const int64_t t = blockIdx.x, units = H / n;
  const int32_t* slots = slot_row + t * top_k;
  for (int64_t u = (int64_t)blockIdx.y * blockDim.x + threadIdx.x; u < units; u += (int64_t)gridDim.y * blockDim.x) {
    Unit<T, kBytes> v, none;
    v.load(x + t * ldx + u * n);
    none.zero();
    for (int j = 0; j < top_k; ++j) {
      const int32_t s = __ldg(slots + j);
      const uint32_t row = s < 0 ? ~s : s;
      if (row < S) (s < 0 ? none : v).store(rows + (int64_t)row * H + u * n);
    }
  }
}

// Every thread sums kU units of the token's row, threads apart, over the slots
// in groups of kJ whose loads are all in flight before the first is used.
// 4096 x 7168 bf16, top-8: 83 us (6.4 TB/s; kJ = 8: 88 us); 3001 x 2047 f32,
// top-4, single elements: 21.4 us (one unit and one slot at a time: 53.7 us).
template <typename T, int kBytes, int kU, int kJ>
__global__ void __launch_bounds__(256)
    combine_kernel(const T* __restrict__ rows, int64_t ld, int64_t H, const int32_t* __restrict__ slot_row,
                   const float* __restrict__ weights, int top_k, uint32_t S, T* __restrict__ out) {
  pdl_wait();
  constexpr int n = Unit<T, kBytes>::n;
  const int64_t t = blockIdx.x, units = H / n;
  for (int64_t u0 = (int64_t)blockIdx.y * blockDim.x * kU + threadIdx.x; u0 - threadIdx.x < units;
       u0 += (int64_t)gridDim.y * blockDim.x * kU) {
    float acc[kU][n];
#pragma unroll
    for (int a = 0; a < kU; ++a)
#pragma unroll
      for (int i = 0; i < n; ++i) acc[a][i] = 0.f;
    for (int j0 = 0; j0 < top_k; j0 += kJ) {
      const T* row[kJ];
      float w[kJ];
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        const int32_t s = j0 + j < top_k ? __ldg(slot_row + t * top_k + j0 + j) : -1;
        const bool live = (uint32_t)s < S;
        row[j] = live ? rows + (int64_t)s * ld : nullptr;
        w[j] = live && weights ? __ldg(weights + t * top_k + j0 + j) : 1.f;
      }
      Unit<T, kBytes> v[kU][kJ];
#pragma unroll
      for (int a = 0; a < kU; ++a)
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
          const int64_t u = u0 + (int64_t)a * blockDim.x;
          if (row[j] && u < units) v[a][j].load(row[j] + u * n);
        }
#pragma unroll
      for (int a = 0; a < kU; ++a)
#pragma unroll
        for (int j = 0; j < kJ; ++j)
          if (row[j]) {
            float f[n];
            v[a][j].floats(f);
#pragma unroll
            for (int i = 0; i < n; ++i) acc[a][i] = fmaf(w[j], f[i], acc[a][i]);
          }
    }
#pragma unroll
    for (int a = 0; a < kU; ++a) {
      const int64_t u = u0 + (int64_t)a * blockDim.x;
      if (u >= units) continue;
      Unit<T, kBytes> o;
      o.round(acc[a]);
      o.store(out + t * H + u * n);
    }
  }
}

constexpr int kGradThreads = 256;

// kWarps warps per slot: the slot's row is read once, w d_out[t] written once,
// and the dot product stays in registers, as 32 kU kWarps partial sums, until
// the end of the row; kU loads of the row in flight per lane.  One warp, which
// needs no barrier, where the slots fill the GPU: the token's other slots are
// the neighbouring warps', so d_out[t] comes from L1 for all but one.  Eight,
// joined in order of the warps, where they do not.
// d_rows may be rows itself: a row belongs to one slot, and a thread reads a
// unit of it before it writes the same one, the only thread to do either.
// 4096 x 7168 bf16, top-8: 149 us (6.7 TB/s, the copy rate; one block per
// token: 182 to 207 us).
template <typename T, int kBytes, int kU, int kWarps>
__global__ void __launch_bounds__(kGradThreads)
    combine_backward_kernel(const T* __restrict__ d_out, int64_t ldd, const T* rows, int64_t ld, int64_t H,
                            const int32_t* __restrict__ slot_row, const float* __restrict__ weights, int top_k,
                            uint32_t S, T* d_rows, float* __restrict__ d_weights) {
  pdl_wait();
  constexpr int n = Unit<T, kBytes>::n, kSlots = kGradThreads / 32 / kWarps;  // slots per block
  __shared__ float joined[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t slot = blockIdx.x * kSlots + warp / kWarps;
  if (slot >= S) return;  // with kWarps = 8 the same for the whole block
  const int first = (warp % kWarps) * 32 + lane, step = 32 * kWarps;
  const int64_t units = H / n;
  const int32_t s = __ldg(slot_row + slot);
  const uint32_t row = s < 0 ? ~s : s;
  const bool live = s >= 0 && row < S, read = live && d_weights;
  const float w = live ? __ldg(weights + slot) : 0.f;
  const T* d_row = d_out + (int64_t)(slot / top_k) * ldd;
  float part[kU];
#pragma unroll
  for (int a = 0; a < kU; ++a) part[a] = 0.f;
  if (row < S) {
    for (int64_t u0 = first; u0 < units; u0 += step * kU) {
      Unit<T, kBytes> d[kU], y[kU];
#pragma unroll
      for (int a = 0; a < kU; ++a) {
        const int64_t u = u0 + step * a;
        if (read && u < units) y[a].template load<false>(rows + (int64_t)row * ld + u * n);
      }
#pragma unroll
      for (int a = 0; a < kU; ++a) {
        const int64_t u = u0 + step * a;
        if (live && u < units) d[a].load(d_row + u * n);
      }
#pragma unroll
      for (int a = 0; a < kU; ++a) {
        const int64_t u = u0 + step * a;
        if (u >= units) continue;
        float f[n];
        if (live) {
          d[a].floats(f);
          if (read) {
            float g[n];
            y[a].floats(g);
#pragma unroll
            for (int i = 0; i < n; ++i) part[a] = fmaf(f[i], g[i], part[a]);
          }
#pragma unroll
          for (int i = 0; i < n; ++i) f[i] *= w;
          d[a].round(f);
        } else {
          d[a].zero();
        }
        d[a].store(d_rows + (int64_t)row * H + u * n);
      }
    }
  }
  if (d_weights) {
    float dot = 0.f;
#pragma unroll
    for (int a = 0; a < kU; ++a) dot += part[a];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(kFull, dot, o);
    if constexpr (kWarps > 1) {
      if (lane == 0) joined[warp] = dot;
      __syncthreads();
      if (warp == 0) {
        dot = 0.f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) dot += joined[i];
      }
    }
    if (lane == 0 && warp % kWarps == 0) d_weights[slot] = dot;
  }
}

// ------------------------------------------------------------------ launches
template <typename F>
q4_status by_dtype(int dtype, F&& f) {
  if (dtype == Q4_F32) return f(float());
  if (dtype == Q4_BF16) return f(__nv_bfloat16());
  return f(__half());
}

// The unit that every row of these matrices can be cut into: their addresses
// and row pitches, and the width H, are multiples of it.
struct Matrix {
  const void* p;
  int64_t pitch;
};
template <typename T>
int unit_bytes(int64_t H, std::initializer_list<Matrix> all) {
  uintptr_t bits = (uintptr_t)(H * sizeof(T));
  for (const Matrix& m : all) bits |= reinterpret_cast<uintptr_t>(m.p) | (uintptr_t)(m.pitch * sizeof(T));
  return bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : (int)sizeof(T);
}
// f with the unit's size as a constant.
template <typename T, typename F>
q4_status by_unit(int bytes, F&& f) {
  if (bytes == 16) return f(std::integral_constant<int, 16>());
  if (bytes == 4) return f(std::integral_constant<int, 4>());
  return f(std::integral_constant<int, (int)sizeof(T)>());
}

// Threads and y blocks for one row of `units` per token: enough blocks to
// fill the GPU when there are few tokens.
inline void row_grid(int64_t tokens, int64_t units, dim3& grid, dim3& block) {
  const int64_t threads = std::min<int64_t>(256, ceil_div(units, 32) * 32);
  const int64_t want = ceil_div((int64_t)num_sms() * 4, tokens);
  const int64_t y = std::max<int64_t>(1, std::min<int64_t>(want, ceil_div(units, threads)));
  grid = dim3((unsigned)tokens, (unsigned)std::min<int64_t>(y, 65535));
  block = dim3((unsigned)threads);
}

}  // namespace

#define Q4_ROUTE_NV(KERNEL, ...)                                                                  \
  (E <= 32 ? launch_pdl(KERNEL<T, 1>, grid, block, 0, stream, __VA_ARGS__)                        \
   : E <= 64 ? launch_pdl(KERNEL<T, 2>, grid, block, 0, stream, __VA_ARGS__)                      \
   : E <= 128 ? launch_pdl(KERNEL<T, 4>, grid, block, 0, stream, __VA_ARGS__)                     \
   : E <= 256 ? launch_pdl(KERNEL<T, 8>, grid, block, 0, stream, __VA_ARGS__)                     \
   : E <= 512 ? launch_pdl(KERNEL<T, 16>, grid, block, 0, stream, __VA_ARGS__)                    \
              : launch_pdl(KERNEL<T, 32>, grid, block, 0, stream, __VA_ARGS__))

q4_status launch_route(const void* logits, int dtype, int64_t tokens, int E, int64_t ld, int top_k, bool over_all,
                       int32_t* ids, float* weights, cudaStream_t stream) {
  const dim3 grid((unsigned)ceil_div(tokens, kRouteWarps)), block(kRouteWarps * kWarp);
  return by_dtype(dtype, [&](auto tag) {
    using T = decltype(tag);
    return Q4_ROUTE_NV(route_kernel, static_cast<const T*>(logits), tokens, E, ld, top_k, (int)over_all, ids,
                       weights, device_status_ptr());
  });
}

q4_status launch_route_backward(const void* logits, int dtype, int64_t tokens, int E, int64_t ld, int top_k,
                                bool over_all, const int32_t* ids, const float* d_weights, void* d_logits,
                                cudaStream_t stream) {
  const dim3 grid((unsigned)ceil_div(tokens, kRouteWarps)), block(kRouteWarps * kWarp);
  return by_dtype(dtype, [&](auto tag) {
    using T = decltype(tag);
    return Q4_ROUTE_NV(route_backward_kernel, static_cast<const T*>(logits), tokens, E, ld, top_k, (int)over_all,
                       ids, d_weights, static_cast<T*>(d_logits));
  });
}

namespace {
// The cluster sort's shape: a warp per 32 slots, up to 16 per block and as many
// as the counts leave room for, then more blocks, then longer parts (device
// time at 256 experts, 16 / 32 warps per block: 1024 slots 4.8 / 6.0 us, 4096
// 5.2 / 7.2, 16384 7.8 / 8.6).  Above kClusterSortSlots the three launches over
// all SMs are faster: 32768 slots 8.2 us against 11.7, 131072 9.9 against 37;
// below it they are slower (4096: 8.4 us) and cost the host two launches more.
struct ClusterSort {
  int warps, blocks, per_warp;
  size_t smem;
};
constexpr size_t kClusterSortSmem = 200 * 1024;
constexpr int64_t kClusterSortSlots = 16384;

ClusterSort cluster_sort(int64_t S, int E) {
  ClusterSort c;
  const int64_t room = (int64_t)(kClusterSortSmem / 4) / (E + 1) - 1;
  const int64_t want = ceil_div(S, 32);
  c.warps = (int)std::max<int64_t>(1, std::min<int64_t>({kClusterWarps, room, want}));
  c.blocks = 1;
  while (c.blocks < kMaxCluster && (int64_t)c.blocks * c.warps < want) c.blocks *= 2;
  c.per_warp = (int)(ceil_div(ceil_div(S, (int64_t)c.blocks * c.warps), 32) * 32);
  c.smem = (size_t)(c.warps + 1) * (E + 1) * sizeof(int32_t);
  return c;
}

q4_status launch_cluster_sort(const ClusterSort& c, const int32_t* ids, int64_t S, int top_k, int E, int32_t* offsets,
                              int32_t* row_token, int32_t* slot_row, cudaStream_t stream) {
  static int attr_done[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return Q4_ERR_CUDA;
  if (!attr_done[dev]) {
    Q4_CUDA_TRY(cudaFuncSetAttribute(sort_cluster_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)kClusterSortSmem));
    attr_done[dev] = 1;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)c.blocks);
  cfg.blockDim = dim3((unsigned)c.warps * 32);
  cfg.dynamicSmemBytes = c.smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)c.blocks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  Q4_CUDA_TRY(cudaLaunchKernelEx(&cfg, sort_cluster_kernel, ids, (int)S, E, top_k, c.per_warp, offsets, row_token,
                                 slot_row));
  return Q4_OK;
}
}  // namespace

// Counts per expert and chunk, then the experts' totals; none where one
// cluster sorts.
size_t moe_sort_workspace_bytes(int64_t S, int64_t E) {
  if (S <= kClusterSortSlots) return 0;
  return (size_t)(E + 1) * (size_t)(ceil_div(S, kSortChunk) + 1) * sizeof(int32_t);
}

q4_status launch_moe_sort(const int32_t* ids, int64_t S, int top_k, int E, int32_t* offsets, int32_t* row_token,
                          int32_t* slot_row, void* ws, cudaStream_t stream) {
  if (S <= kClusterSortSlots)
    return launch_cluster_sort(cluster_sort(S, E), ids, S, top_k, E, offsets, row_token, slot_row, stream);
  const int chunks = (int)ceil_div(S, kSortChunk);
  int32_t* hist = static_cast<int32_t*>(ws);
  int32_t* total = hist + (int64_t)(E + 1) * chunks;
  const size_t row = (size_t)(E + 1) * sizeof(int32_t);
  q4_status st = launch_pdl(sort_count_kernel, chunks, kSortThreads, row, stream, ids, S, E, chunks, hist);
  if (st != Q4_OK) return st;
  st = launch_pdl(sort_scan_kernel, E + 1, kSortThreads, 0, stream, chunks, hist, total);
  if (st != Q4_OK) return st;
  return launch_pdl(sort_place_kernel, chunks, kSortThreads, (kSortWarps + 1) * row, stream, ids, S, E, top_k,
                    chunks, hist, total, offsets, row_token, slot_row);
}

q4_status launch_dispatch(const void* x, int dtype, int64_t tokens, int64_t H, int64_t ldx, const int32_t* slot_row,
                          int top_k, void* rows, cudaStream_t stream) {
  return by_dtype(dtype, [&](auto tag) {
    using T = decltype(tag);
    return by_unit<T>(unit_bytes<T>(H, {{x, ldx}, {rows, H}}), [&](auto bytes) {
      constexpr int B = decltype(bytes)::value;
      dim3 grid, block;
      row_grid(tokens, H * (int64_t)sizeof(T) / B, grid, block);
      return launch_pdl(dispatch_kernel<T, B>, grid, block, 0, stream, static_cast<const T*>(x), ldx, H, slot_row,
                        top_k, (uint32_t)(tokens * top_k), static_cast<T*>(rows));
    });
  });
}

q4_status launch_combine(const void* rows, int dtype, int64_t tokens, int64_t H, int64_t ld, const int32_t* slot_row,
                         const float* weights, int top_k, void* out, cudaStream_t stream) {
  return by_dtype(dtype, [&](auto tag) {
    using T = decltype(tag);
    return by_unit<T>(unit_bytes<T>(H, {{rows, ld}, {out, H}}), [&](auto bytes) {
      constexpr int B = decltype(bytes)::value, per = B == 16 ? 1 : 4;  // units per thread
      const int64_t units = H * (int64_t)sizeof(T) / B;
      const int64_t threads = std::min<int64_t>(256, ceil_div(ceil_div(units, per), 32) * 32);
      const dim3 grid((unsigned)tokens, (unsigned)std::min<int64_t>(65535, ceil_div(units, threads * per)));
      return launch_pdl(combine_kernel<T, B, per, 4>, grid, dim3((unsigned)threads), 0, stream,
                        static_cast<const T*>(rows), ld, H, slot_row, weights, top_k, (uint32_t)(tokens * top_k),
                        static_cast<T*>(out));
    });
  });
}

q4_status launch_combine_backward(const void* d_out, int dtype, int64_t tokens, int64_t H, int64_t ldd,
                                  const void* rows, int64_t ld, const int32_t* slot_row, const float* weights,
                                  int top_k, void* d_rows, float* d_weights, cudaStream_t stream) {
  return by_dtype(dtype, [&](auto tag) {
    using T = decltype(tag);
    const Matrix read = d_weights ? Matrix{rows, ld} : Matrix{d_out, ldd};
    return by_unit<T>(unit_bytes<T>(H, {{d_out, ldd}, {d_rows, H}, read}), [&](auto bytes) {
      constexpr int B = decltype(bytes)::value;
      constexpr int U = B == 16 ? 4 : 8;
      const uint32_t S = (uint32_t)(tokens * top_k);
      // warps per slot; 8 against 1 at 7168 wide: 128 slots 2.1 / 5.9 us, 512 3.1 / 6.0, 1024 5.1 / 6.1 (at
      // 2048 wide 3.5 / 2.8), 2048 8.2 / 7.5
      const int warps = S <= 4u * (uint32_t)num_sms() ? 8 : 1;
      return launch_pdl(warps == 8 ? combine_backward_kernel<T, B, U, 8> : combine_backward_kernel<T, B, U, 1>,
                        (unsigned)ceil_div((int64_t)S * warps, kGradThreads / 32), kGradThreads, 0, stream,
                        static_cast<const T*>(d_out), ldd, static_cast<const T*>(rows), ld, H, slot_row, weights, top_k,
                        S, static_cast<T*>(d_rows), d_weights);
    });
  });
}

}  // namespace q4
