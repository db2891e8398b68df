// Root-mean-square norm with the residual's addition, its result kept in 16 or
// 32 bits or written in the 8-bit forms that the products read.
//
//   h = x + residual,  rstd = 1 / sqrt(mean(h^2) + eps),  y = h rstd w
//   FP8:  per row and 128 columns s = max(amax |y|, 1e-12) / 448, codes E4M3(y / s)
//   INT8: per row s = max(amax |y|, 1e-12) / 127, codes rint(y / s)
// Everything between the loads and the stores is FP32: h and y are rounded once
// each, and y / s is taken from the unrounded h (y / s = (h w) (rstd / s)).
// amax |h w| needs no rstd, so the row's sum of squares and its largest
// magnitude are reduced together: one exchange between the warps per row.
//
// HBM-bound: every row is read once and stays in registers, 16 lanes per block
// of 128 columns, 8 columns per lane (Piece); `group` threads hold a row, kC
// pieces each.  What registers can hold in flight (32 KB per SM) is too little for
// HBM, so where there are many rows they come through a ring in shared memory,
// filled by bulk copies some rows ahead.
//
// Measured: 8192 x 8192 bf16 with residual to FP8 75.6 us (6.2 TB/s), to bf16 87.5
// (6.1 TB/s); 8192 x 4096 to INT8 41.6 (5.7 TB/s); 4096 x 7168 f16 without residual to
// INT8 22.6 (3.9 TB/s: latency of a row's chain, wait to codes, of which 16 warps per SM
// have one each under way; half of the issue slots are free); 3001 x 2047 FP32
// 18.2 (5.4 TB/s); 8192 x 1411 bf16 to FP8 31.5 (2.6 TB/s: single elements); 4 x 7168
// 3.1 (launch and one row's latency); 256 x 8192 to FP8 6.1, 1000 x 4096 to INT8 7.8;
// 2048 x 32768 112 (4.8 TB/s, no ring).  FP32 weights of 16-bit rows are read for every
// row: 8192 x 8192 to FP8 86.0, 4096 x 7168 to INT8 34.5.
#include "rows.cuh"

namespace q4 {
namespace {

__device__ __forceinline__ uint2 e4m3x8(const float (&v)[8], float f) {
  return make_uint2(e4m3x2(v[0] * f, v[1] * f) | e4m3x2(v[2] * f, v[3] * f) << 16,
                    e4m3x2(v[4] * f, v[5] * f) | e4m3x2(v[6] * f, v[7] * f) << 16);
}

// A row of h = x + residual in v: reduced, scaled by the weights and written.  H is
// 0 for a row that is not there.  kWhole: every piece lies inside the row, which is
// there (a fifth fewer instructions, which bound these kernels beside HBM).
template <typename T, bool kVec, int kC, int kForm, bool kWhole, typename Weights, typename AfterReduce>
__device__ __forceinline__ void norm_row(const NormArgs& a, const Place& pl, int64_t row, int H, float inv_H, float (&v)[kC][8],
                                         Exchange& ex, int buf, int* status, Weights&& weights, AfterReduce&& after_reduce) {
  using P = Piece<T, kVec>;
  const int64_t start = row * a.H;
  auto cols = [&](int i) { return kWhole ? 128 : pl.cols(i, H); };
  float sum = 0.f, top = 0.f;
  if (a.h) {
    T* h = static_cast<T*>(a.h) + start;
#pragma unroll
    for (int i = 0; i < kC; ++i) P::store(h + pl.at(i), pl.l, cols(i), v[i]);
  }
#pragma unroll
  for (int i = 0; i < kC; ++i) {
    float w[8];
    weights(i, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      sum = fmaf(v[i][j], v[i][j], sum);
      v[i][j] *= w[j];
      if (kForm == Q4_NORM_INT8) top = max_nan(top, fabsf(v[i][j]));
    }
  }
  const float2 r = group_reduce<kForm == Q4_NORM_INT8>(sum, top, pl.group, ex, buf);
  after_reduce();
  const float rstd = rsqrtf(fmaf(r.x, inv_H, a.eps));  // within 2 ulp
  if (pl.t == 0 && H) {
    if (a.rstd) a.rstd[row] = rstd;
    if (nonfinite(r.x)) latch_status(status, Q4_ERR_NONFINITE);
  }
  if constexpr (kForm == Q4_NORM_INT8) {
    // the codes are rint(h w f); where the scale is not the least one, f = rstd / s =
    // 127 / amax |h w| needs neither rstd nor s and their roundings
    const float s = max_nan(r.y * rstd, 1e-12f) * (1.f / 127.f);
    const float f = r.y * rstd > 1e-12f ? __fdiv_rn(127.f, r.y) : __fdiv_rn(rstd, s);
    if (pl.t == 0 && H) {
      a.scales[row] = s;
      if (nonfinite(s)) latch_status(status, Q4_ERR_NONFINITE);
    }
    uint8_t* codes = a.codes + start;
#pragma unroll
    for (int i = 0; i < kC; ++i) P::store_codes(codes + pl.at(i), pl.l, cols(i), int8x8(v[i], f));
  }
  if constexpr (kForm == Q4_NORM_FP8) {
    uint8_t* codes = a.codes + start;
    float* scales = a.scales + row * ((a.H + 127) / 128);
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      float m = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max_nan(m, fabsf(v[i][j]));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float s = max_nan(m * rstd, 1e-12f) * (1.f / 448.f);
      // 448 / m, as 7 / (m / 64): __fdividef gives 0 for divisors above 2^126
      const float f = m * rstd > 1e-12f ? __fdividef(7.f, m * 0x1p-6f) : __fdividef(rstd, s);
      P::store_codes(codes + pl.at(i), pl.l, cols(i), e4m3x8(v[i], f));
      if (pl.l == 0 && cols(i) > 0) {
        scales[pl.block(i)] = s;
        if (nonfinite(s)) latch_status(status, Q4_ERR_NONFINITE);
      }
    }
  }
  if (a.y) {
    T* out = static_cast<T*>(a.y) + start;
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = v[i][j] * rstd;
      P::store(out + pl.at(i), pl.l, cols(i), y);
    }
  }
}

// A row's pieces x (+ res) into v.
template <typename T, bool kVec, int kC, bool kWhole>
__device__ __forceinline__ void load_row(const T* x, const T* res, bool add, const Place& pl, int H, float (&v)[kC][8]) {
  using P = Piece<T, kVec>;
#pragma unroll
  for (int i = 0; i < kC; ++i) {
    P px;
    px.load(x + pl.at(i), pl.l, kWhole ? 128 : pl.cols(i, H));
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = px.at(j);
  }
  if (!add) return;
#pragma unroll
  for (int i = 0; i < kC; ++i) {
    P pr;
    pr.load(res + pl.at(i), pl.l, kWhole ? 128 : pl.cols(i, H));
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] += pr.at(j);
  }
}

// Rows straight from global memory: few rows, or long ones that the ring has no room for.
template <typename T, bool kVec, int kC, int kForm>
__global__ void __launch_bounds__(max_threads(kC))
    norm_kernel(const NormArgs a, int group, int* status) {
  pdl_wait();
  __shared__ Exchange ex;
  exchange_init(ex);
  __syncthreads();
  const Place pl(group);
  const int width = (int)a.H;
  const float inv_H = 1.f / (float)width;
  auto weights = [&](int i, float (&f)[8]) {
    load_weights<T, kVec>(a.weight, a.w_dtype == Q4_F32, pl.at(i), pl.l, pl.cols(i, width), f);
  };
  int buf = 0;
  for (int64_t base = (int64_t)blockIdx.x * pl.per_block; base < a.rows; base += (int64_t)gridDim.x * pl.per_block, buf ^= 1) {
    const int64_t row = base + pl.sub;
    const int H = row < a.rows ? width : 0;
    float v[kC][8];
    load_row<T, kVec, kC, false>(static_cast<const T*>(a.x) + row * a.ldx, static_cast<const T*>(a.residual) + row * a.ld_residual,
                                 a.residual != nullptr, pl, H, v);
    norm_row<T, kVec, kC, kForm, false>(a, pl, row, H, inv_H, v, ex, buf, status, weights, [] {});
  }
}

template <typename T, bool kVec, int kC, int kForm, int kThreads>
__global__ void __launch_bounds__(kThreads, resident_blocks(kVec, kThreads, false)) norm_ring_kernel(const NormArgs a, int group, const RingArgs r) {
  extern __shared__ __align__(128) uint8_t stage_smem[];
  __shared__ Ring ring;
  __shared__ Exchange ex;
  ring_init(ring, r, ex);
  pdl_wait();
  const Place pl(group);
  const int width = (int)a.H;
  const float inv_H = 1.f / (float)width;
  const void* const mat[2] = {a.x, a.residual};
  const int64_t pitch[2] = {a.ldx * (int64_t)sizeof(T), a.ld_residual * (int64_t)sizeof(T)};
  const int64_t step = (int64_t)gridDim.x * pl.per_block, base0 = (int64_t)blockIdx.x * pl.per_block;
  if (threadIdx.x == 0)
    for (int s = 0; s < r.stages; ++s)
      ring_fill<kVec>(ring, r, smem_u32(stage_smem), s, mat, pitch, base0 + s * step, a.rows, pl.per_block);
  const HeldWeights<T, kVec, kC> w(a.weight, a.w_dtype, pl, width);
  int stage = 0, buf = 0;
  uint32_t phase = 0;
  auto rows = [&](auto tag) {
    constexpr bool kWhole = decltype(tag)::value;
    auto weights = [&](int i, float (&f)[8]) { w.template get<kWhole>(pl, width, i, f); };
    for (int64_t base = base0; base < a.rows; base += step, buf ^= 1) {
      const int64_t row = base + pl.sub;
      const int H = kWhole || row < a.rows ? width : 0;
      mbar_wait(smem_u32(&ring.full[stage]), phase, r.ctl, &ring.abort);
      float v[kC][8];
      if (!kVec && read_in_place(row, a.rows, r.edge)) {
        load_row<T, kVec, kC, kWhole>(static_cast<const T*>(a.x) + row * a.ldx,
                                      static_cast<const T*>(a.residual) + row * a.ld_residual, a.residual != nullptr, pl, H, v);
      } else {
        const uint8_t* st = stage_smem + stage * r.stage_bytes;
        load_row<T, kVec, kC, kWhole>(ring_row<kVec, T>(st, r, 0, pl, a.x, pitch[0], row),
                                      ring_row<kVec, T>(st, r, 1, pl, a.residual, pitch[1], row), a.residual != nullptr, pl, H, v);
      }
      norm_row<T, kVec, kC, kForm, kWhole>(
          a, pl, row, H, inv_H, v, ex, buf, r.ctl.status, weights,
          [&] {  // every thread has read the stage: the next rows may come
            if (pl.group <= 32) __syncthreads();
            if (threadIdx.x == 0 && ring_over(ring, stage, phase))
              ring_fill<kVec>(ring, r, smem_u32(stage_smem), stage, mat, pitch, base + r.stages * step, a.rows, pl.per_block);
          });
      if (++stage == r.stages) stage = 0, phase ^= 1;
    }
  };
  if constexpr (kVec && kC == 4) {
    // (not where FP8 codes and h are written: 8192 x 8192 84.6 us instead of 78.1;
    // without a residual 8192 x 2048 15.6 instead of 17.4)
    if ((kForm != Q4_NORM_FP8 || !a.residual) && w.held && pl.whole(kC, width) && a.rows % pl.per_block == 0)
      rows(std::true_type());
    else
      rows(std::false_type());
  } else {
    rows(std::false_type());
  }
  ring_end(ring, r);
}

template <typename T, bool kVec, int kC, int kForm, int kThreads>
q4_status launch_norm_ring(const NormArgs& a, const Shape& s, cudaStream_t stream) {
  static std::atomic<int> ready[64];
  const auto kernel = norm_ring_kernel<T, kVec, kC, kForm, kThreads>;
  const q4_status st = allow_smem(kernel, ready);
  if (st != Q4_OK) return st;
  return launch_pdl(kernel, s.grid, s.threads, (size_t)s.stages * s.stage_bytes, stream, a, s.group,
                    ring_of(s, kVec, a.H * (int64_t)sizeof(T)));
}

template <typename T, int kC, int kForm>
q4_status launch_norm_form(const NormArgs& a, const Shape& s, bool vec, cudaStream_t stream) {
  if (s.stages) {
    if constexpr (kC == 2)
      if (!vec) return launch_norm_ring<T, false, kC, kForm, 256>(a, s, stream);
    if constexpr (kC == 4)
      if (s.threads > 256) return launch_norm_ring<T, true, kC, kForm, 512>(a, s, stream);
    if constexpr (kC <= 4) return launch_norm_ring<T, true, kC, kForm, 256>(a, s, stream);
  }
  if constexpr (kC != 2)
    return launch_pdl(vec ? norm_kernel<T, true, kC, kForm> : norm_kernel<T, false, kC, kForm>, s.grid, s.threads, 0, stream, a,
                      s.group, device_status_ptr());
  return Q4_ERR_UNSUPPORTED_SHAPE;  // not reached: two pieces are for rings
}

}  // namespace

q4_status launch_norm(const NormArgs& a, int dtype, int form, cudaStream_t stream) {
  const int size = dtype == Q4_F32 ? 4 : 2;
  const bool vec = a.H % 8 == 0 && a.ldx * size % 16 == 0 && (!a.residual || a.ld_residual * size % 16 == 0) && mult(a.x, 16) &&
                   mult(a.residual, 16) && mult(a.h, 16) && mult(a.y, 16) && mult(a.codes, 8) && mult(a.weight, 16);
  const Shape s = shape_of(a.rows, a.H, a.residual ? 2 : 1, size, vec, false);
  return by_dtype(dtype, [&](auto tag) {
    using T = decltype(tag);
    return by_pieces(s.C, [&](auto c) {
      constexpr int C = decltype(c)::value;
      if (form == Q4_NORM_FP8) return launch_norm_form<T, C, Q4_NORM_FP8>(a, s, vec, stream);
      if (form == Q4_NORM_INT8) return launch_norm_form<T, C, Q4_NORM_INT8>(a, s, vec, stream);
      return launch_norm_form<T, C, Q4_NORM_PLAIN>(a, s, vec, stream);
    });
  });
}

}  // namespace q4
