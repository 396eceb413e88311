// norm.cu -- pw_add_rms_norm: residual addition, root-mean-square norm and an
// optional 8-bit output with scales, in one pass over the rows.
//
//   h = x + r                        (fp32, each input widened exactly)
//   r_out = round(h)                 (to the residual output's type)
//   y = h * (mean(h^2) + eps)^-1/2 * w
//   bf16 output: round(y).  e4m3 output, per row or per 128 columns:
//   s = max(max|y| / 448, 2^-126), q = e4m3(y / s).
//
// The row stays in registers between its two uses, so every input is read
// once and every output written once.  The sum of squares and max|h w| come
// from the same reduction (|y| = |h w| * rstd with rstd > 0, so max|y| needs no
// pass of its own): one block barrier a row.  All statistics are fp32.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <cfloat>
#include <cmath>
#include <type_traits>

#include "pw_internal.h"

namespace pw {
namespace {

constexpr int kNormThreads = 1024;  // most threads of a row
constexpr int kNormMaxH = 32768;
constexpr float kE4m3Max = 448.0f;
constexpr float kScaleMin = 1.17549435e-38f;  // 2^-126: keeps y / s finite for rows of zeros

enum NormOut { kOutBf16 = 0, kOutE4m3Row = 1, kOutE4m3Group = 2 };
constexpr int kGroup = 128;  // columns of a scale group

struct NormParams {
  const void* x;
  const void* res;
  const void* w;
  void* res_out;
  void* y;
  float* scales;
  int64_t x_ld, res_ld, res_out_ld, y_ld;
  int T, H, n_groups, tpr, w_f32;  // tpr: threads of a row
  float eps, inv_h;
};

struct None {};

// N consecutive elements as they lie in memory, N = 8 (16-byte loads) or 1.
template <typename T, int N>
struct Raw;
template <>
struct Raw<__nv_bfloat16, 8> {
  uint4 v;
  __device__ void load(const void* p, int64_t i) {
    v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
  }
  __device__ void zero() { v = make_uint4(0, 0, 0, 0); }
  __device__ float get(int k) const {
    const uint32_t u = k < 2 ? v.x : k < 4 ? v.y : k < 6 ? v.z : v.w;
    return __uint_as_float((k & 1) ? (u & 0xffff0000u) : (u << 16));
  }
};
template <>
struct Raw<float, 8> {
  float4 a, b;
  __device__ void load(const void* p, int64_t i) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    a = q[0];
    b = q[1];
  }
  __device__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ float get(int k) const {
    const float4& c = k < 4 ? a : b;
    const int j = k & 3;
    return j == 0 ? c.x : j == 1 ? c.y : j == 2 ? c.z : c.w;
  }
};
template <>
struct Raw<__nv_bfloat16, 1> {
  uint16_t v;
  __device__ void load(const void* p, int64_t i) { v = static_cast<const uint16_t*>(p)[i]; }
  __device__ void zero() { v = 0; }
  __device__ float get(int) const { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
};
template <>
struct Raw<float, 1> {
  float v;
  __device__ void load(const void* p, int64_t i) { v = static_cast<const float*>(p)[i]; }
  __device__ void zero() { v = 0.f; }
  __device__ float get(int) const { return v; }
};
template <int N>
struct Raw<None, N> {
  __device__ void load(const void*, int64_t) {}
  __device__ void zero() {}
  __device__ float get(int) const { return 0.f; }
};

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <int N>
__device__ __forceinline__ void store_bf16(void* p, int64_t i, const float* v) {
  uint16_t* q = static_cast<uint16_t*>(p) + i;
  if constexpr (N == 8)
    *reinterpret_cast<uint4*>(q) = make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]),
                                              bf16x2(v[4], v[5]), bf16x2(v[6], v[7]));
  else
    *q = static_cast<uint16_t>(bf16x2(v[0], 0.f) & 0xffffu);
}
template <int N>
__device__ __forceinline__ void store_f32(void* p, int64_t i, const float* v) {
  float* q = static_cast<float*>(p) + i;
  if constexpr (N == 8) {
    reinterpret_cast<float4*>(q)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(q)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *q = v[0];
  }
}
// two floats to e4m3, lo in the low byte; NaN stays NaN, |v| > 448 saturates
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
template <int N>
__device__ __forceinline__ void store_e4m3(void* p, int64_t i, const float* v) {
  uint8_t* q = static_cast<uint8_t*>(p) + i;
  if constexpr (N == 8)
    *reinterpret_cast<uint2*>(q) = make_uint2(e4m3x2(v[0], v[1]) | (e4m3x2(v[2], v[3]) << 16),
                                              e4m3x2(v[4], v[5]) | (e4m3x2(v[6], v[7]) << 16));
  else
    *q = static_cast<uint8_t>(e4m3x2(v[0], 0.f) & 0xffu);
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// (sum of a, NaN-keeping max of b) over the row's threads, the same in all of
// them.  Rows of one warp need no barrier; wider rows own their block, and the
// two halves of `part` alternate from row to row, so one barrier is enough.
__device__ __forceinline__ void row_reduce(float& a, float& b, int tpr, float2* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b = max_nan(b, __shfl_xor_sync(0xffffffffu, b, o));
  }
  if (tpr == 32) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = tpr >> 5;
  if (lane == 0) part[warp] = make_float2(a, b);
  __syncthreads();
  const float2 v = lane < nw ? part[lane] : make_float2(0.f, 0.f);
  a = v.x;
  b = v.y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b = max_nan(b, __shfl_xor_sync(0xffffffffu, b, o));
  }
}

// One row per tpr threads, M vectors of N columns a thread.  Vector v of a row
// belongs to thread v % tpr: a warp's accesses are contiguous.
// One block an SM is named as the least: without it the compiler takes 32
// registers for some forms that spill anyway (above 8192 columns), in the hope
// of two (2048 x 20480 bf16: 184 us against 100; 2048 x 14335: 610 against 522).
template <typename XT, typename RT, int OUT, int N, int M>
__global__ void __launch_bounds__(kNormThreads, 1) norm_kernel(const NormParams p) {
  extern __shared__ float gmax[];  // N = 1 group scales: [2][M * tpr / 32] warp maxima
  __shared__ float2 part[2][32];
  const int tpr = p.tpr, lane_r = threadIdx.x % tpr, rows_blk = blockDim.x / tpr;
  pdl_wait();
  // the weights stay in registers over the rows where there is room
  constexpr bool kHold = N * M <= 8;
  float wv[kHold ? M : 1][N];
  auto load_w = [&](int j, float* w) {
    const int c = (j * tpr + lane_r) * N;
    Raw<float, N> rf;
    Raw<__nv_bfloat16, N> rb;
    rf.zero();
    if (c < p.H) {
      if (p.w_f32) {
        rf.load(p.w, c);
      } else {
        rb.load(p.w, c);
#pragma unroll
        for (int k = 0; k < N; ++k) w[k] = rb.get(k);
        return;
      }
    }
#pragma unroll
    for (int k = 0; k < N; ++k) w[k] = rf.get(k);
  };
  if constexpr (kHold) {
#pragma unroll
    for (int j = 0; j < M; ++j) load_w(j, wv[j]);
  }
  // the next row's loads are in flight while a row is reduced and written
  Raw<XT, N> rx[M];
  Raw<RT, N> rr[M];
  auto load_row = [&](int64_t row) {
#pragma unroll
    for (int j = 0; j < M; ++j) {
      const int c = (j * tpr + lane_r) * N;
      if (row < p.T && c < p.H) {
        rx[j].load(p.x, row * p.x_ld + c);
        rr[j].load(p.res, row * p.res_ld + c);
      } else {
        rx[j].zero();
        rr[j].zero();
      }
    }
  };
  int parity = 0;
  const int64_t row_step = static_cast<int64_t>(gridDim.x) * rows_blk;
  int64_t row = static_cast<int64_t>(blockIdx.x) * rows_blk + threadIdx.x / tpr;
  load_row(row);
  for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * rows_blk; row0 < p.T;
       row0 += row_step, row += row_step, parity ^= 1) {
    const bool live = row < p.T;  // a whole warp agrees: rows sharing a block are a warp each
    float h[M][N];
#pragma unroll
    for (int j = 0; j < M; ++j)
#pragma unroll
      for (int k = 0; k < N; ++k) h[j][k] = rx[j].get(k) + rr[j].get(k);
    load_row(row + row_step);
    if constexpr (!std::is_same<RT, None>::value) {
      if (p.res_out && live) {
#pragma unroll
        for (int j = 0; j < M; ++j) {
          const int c = (j * tpr + lane_r) * N;
          if (c >= p.H) continue;
          if constexpr (std::is_same<RT, float>::value)
            store_f32<N>(p.res_out, row * p.res_out_ld + c, h[j]);
          else
            store_bf16<N>(p.res_out, row * p.res_out_ld + c, h[j]);
        }
      }
    }
    float ss = 0.f, mx = 0.f, gm[M];
    auto stats = [&]() {
      ss = mx = 0.f;
#pragma unroll
      for (int j = 0; j < M; ++j) {
        gm[j] = 0.f;
        float* w = wv[kHold ? j : 0];
        if constexpr (!kHold && OUT != kOutBf16) load_w(j, w);
#pragma unroll
        for (int k = 0; k < N; ++k) {
          ss = fmaf(h[j][k], h[j][k], ss);
          if constexpr (OUT != kOutBf16) gm[j] = max_nan(gm[j], fabsf(h[j][k] * w[k]));
        }
        if constexpr (OUT != kOutBf16) mx = max_nan(mx, gm[j]);
      }
    };
    auto group_max = [&]() {
      if constexpr (OUT == kOutE4m3Group) {
        if constexpr (N == 8) {  // 16 lanes hold a group
#pragma unroll
          for (int j = 0; j < M; ++j)
#pragma unroll
            for (int o = 8; o > 0; o >>= 1)
              gm[j] = max_nan(gm[j], __shfl_xor_sync(0xffffffffu, gm[j], o));
        } else {  // four warps hold a group; read behind row_reduce's barrier
#pragma unroll
          for (int j = 0; j < M; ++j) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
              gm[j] = max_nan(gm[j], __shfl_xor_sync(0xffffffffu, gm[j], o));
            if ((threadIdx.x & 31) == 0)
              gmax[(parity * M + j) * (tpr >> 5) + (lane_r >> 5)] = gm[j];
          }
        }
      }
    };
    stats();
    group_max();
    row_reduce(ss, mx, tpr, part[parity]);
    float rstd = 1.0f / sqrtf(fmaf(ss, p.inv_h, p.eps));
    // Out of fp32's range, the same for the row: the squares, or (8-bit forms)
    // the largest |h w|, which only large weights can take there.  The row then
    // becomes h / rms, where 1 / rms alone could be subnormal.
    if (isinf(ss) || (OUT != kOutBf16 && isinf(mx))) {
      float f = 1.0f;
      if (isinf(ss)) {
        // once more on h * f, f = 2^-80, whose squares cannot (|h| < 2^128,
        // 2^15 columns).  With the mean scaled by f^2, eps is too: a row that
        // only just overflows has a scaled mean near 2^-47, far below a usual
        // eps as it stands.
        f = 8.271806125530277e-25f;
        ss = 0.f;
#pragma unroll
        for (int j = 0; j < M; ++j)
#pragma unroll
          for (int k = 0; k < N; ++k) ss = fmaf(h[j][k] * f, h[j][k] * f, ss);
        parity ^= 1;
        row_reduce(ss, mx, tpr, part[parity]);
        rstd = 1.0f / sqrtf(fmaf(ss, p.inv_h, p.eps * f * f));
      }
#pragma unroll
      for (int j = 0; j < M; ++j)
#pragma unroll
        for (int k = 0; k < N; ++k) h[j][k] = h[j][k] * rstd * f;
      rstd = 1.0f;
      if constexpr (OUT != kOutBf16) {
        parity ^= 1;
        stats();
        group_max();
        row_reduce(ss, mx, tpr, part[parity]);
      }
    }
    if (!live) continue;
    if constexpr (OUT == kOutE4m3Row) {
      const float s = max_nan(mx * rstd / kE4m3Max, kScaleMin);
      if (lane_r == 0) p.scales[row] = s;
      const float inv = 1.0f / s;
#pragma unroll
      for (int j = 0; j < M; ++j) {
        const int c = (j * tpr + lane_r) * N;
        if (c >= p.H) continue;
        float q[N];
        float* w = wv[kHold ? j : 0];
        if constexpr (!kHold) load_w(j, w);
#pragma unroll
        for (int k = 0; k < N; ++k) q[k] = h[j][k] * rstd * w[k] * inv;
        store_e4m3<N>(p.y, row * p.y_ld + c, q);
      }
    } else if constexpr (OUT == kOutE4m3Group) {
#pragma unroll
      for (int j = 0; j < M; ++j) {
        const int c = (j * tpr + lane_r) * N;
        if constexpr (N == 1) {
          const int w0 = (lane_r >> 5) & ~3;
          const float* g = gmax + (parity * M + j) * (tpr >> 5) + w0;
          gm[j] = max_nan(max_nan(g[0], g[1]), max_nan(g[2], g[3]));
        }
        if (c >= p.H) continue;
        const float s = max_nan(gm[j] * rstd / kE4m3Max, kScaleMin);
        if (c % kGroup == 0) p.scales[row * p.n_groups + c / kGroup] = s;
        const float inv = 1.0f / s;
        float q[N];
        float* w = wv[kHold ? j : 0];
        if constexpr (!kHold) load_w(j, w);
#pragma unroll
        for (int k = 0; k < N; ++k) q[k] = h[j][k] * rstd * w[k] * inv;
        store_e4m3<N>(p.y, row * p.y_ld + c, q);
      }
    } else {
#pragma unroll
      for (int j = 0; j < M; ++j) {
        const int c = (j * tpr + lane_r) * N;
        if (c >= p.H) continue;
        float q[N];
        float* w = wv[kHold ? j : 0];
        if constexpr (!kHold) load_w(j, w);
#pragma unroll
        for (int k = 0; k < N; ++k) q[k] = h[j][k] * rstd * w[k];
        store_bf16<N>(p.y, row * p.y_ld + c, q);
      }
    }
  }
}

template <typename XT, typename RT, int OUT, int N, int M>
cudaError_t launch_shape(NormParams p, int n_sm, cudaStream_t s) {
  const int vecs = (p.H + N * M - 1) / (N * M);
  // scalar group scales are shared by four whole warps
  const int unit = (N == 1 && OUT == kOutE4m3Group) ? 128 : 32;
  p.tpr = (vecs + unit - 1) / unit * unit;
  const int rows_blk = p.tpr == 32 ? 4 : 1;
  const int threads = p.tpr * rows_blk;
  int64_t grid = (static_cast<int64_t>(p.T) + rows_blk - 1) / rows_blk;
  const int64_t most = static_cast<int64_t>(n_sm) * (kNormThreads / threads);
  if (grid > most) grid = most;
  const size_t smem = (N == 1 && OUT == kOutE4m3Group) ? sizeof(float) * 2 * M * (p.tpr >> 5) : 0;
  return launch_pdl(norm_kernel<XT, RT, OUT, N, M>, dim3(static_cast<unsigned>(grid)), dim3(threads),
                    smem, s, p);
}

template <typename XT, typename RT, int OUT>
cudaError_t launch_out(const NormParams& p, bool vec, int n_sm, cudaStream_t s) {
  if (vec) {
    if (p.H <= 8 * kNormThreads) return launch_shape<XT, RT, OUT, 8, 1>(p, n_sm, s);
    if (p.H <= 16 * kNormThreads) return launch_shape<XT, RT, OUT, 8, 2>(p, n_sm, s);
    return launch_shape<XT, RT, OUT, 8, 4>(p, n_sm, s);
  }
  if (p.H <= 8 * kNormThreads) return launch_shape<XT, RT, OUT, 1, 8>(p, n_sm, s);
  return launch_shape<XT, RT, OUT, 1, 32>(p, n_sm, s);
}

template <typename XT, typename RT>
cudaError_t launch_types(const NormParams& p, int out, bool vec, int n_sm, cudaStream_t s) {
  switch (out) {
    case kOutBf16: return launch_out<XT, RT, kOutBf16>(p, vec, n_sm, s);
    case kOutE4m3Row: return launch_out<XT, RT, kOutE4m3Row>(p, vec, n_sm, s);
    default: return launch_out<XT, RT, kOutE4m3Group>(p, vec, n_sm, s);
  }
}

template <typename XT>
cudaError_t launch_x(const NormParams& p, int res_type, int out, bool vec, int n_sm,
                     cudaStream_t s) {
  if (!p.res) return launch_types<XT, None>(p, out, vec, n_sm, s);
  if (res_type == PW_F32) return launch_types<XT, float>(p, out, vec, n_sm, s);
  return launch_types<XT, __nv_bfloat16>(p, out, vec, n_sm, s);
}

int type_bytes(int type) { return type == PW_F32 ? 4 : type == PW_E4M3 ? 1 : 2; }
bool aligned_to(const void* p, int bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}
// 8-column accesses of this matrix are aligned (up to 16 bytes each)
bool vec_ok(const void* p, int64_t ld, int type) {
  return !p || (aligned_to(p, type == PW_E4M3 ? 8 : 16) && ld % (type == PW_F32 ? 4 : 8) == 0);
}

}  // namespace
}  // namespace pw

extern "C" pw_status_t pw_add_rms_norm(const void* d_x, int32_t x_type, int64_t x_stride,
                                       const void* d_residual, int32_t residual_type,
                                       int64_t residual_stride, const void* d_weight,
                                       int32_t weight_type, float eps, int32_t T, int32_t H,
                                       void* d_residual_out, int64_t residual_out_stride,
                                       void* d_y, int32_t y_type, int64_t y_stride,
                                       float* d_scales, int32_t scale_group, pw_stream_t stream) {
  using namespace pw;
  auto bad = [](const char* msg) { return record_error(PW_ERR_INVALID_ARG, msg); };
  if (T < 0 || H < 1) return bad("pw_add_rms_norm: need T >= 0 and H >= 1");
  if (H > kNormMaxH) return record_error(PW_ERR_UNSUPPORTED, "pw_add_rms_norm: H above 32768");
  if ((x_type != PW_BF16 && x_type != PW_F32) || (weight_type != PW_BF16 && weight_type != PW_F32) ||
      (d_residual && residual_type != PW_BF16 && residual_type != PW_F32))
    return bad("pw_add_rms_norm: x, residual and weight are PW_BF16 or PW_F32");
  if (y_type != PW_BF16 && y_type != PW_E4M3)
    return bad("pw_add_rms_norm: y is PW_BF16 or PW_E4M3");
  if (scale_group != 0 && scale_group != kGroup)
    return bad("pw_add_rms_norm: scale_group is 0 (a scale per row) or 128");
  // below 2^-126 the squares that matter beside eps would be subnormal, and the
  // mean good to a few bits only
  if (!(eps >= FLT_MIN) || !std::isfinite(eps))
    return bad("pw_add_rms_norm: eps must be positive (2^-126 at least) and finite");
  if (d_residual_out && !d_residual)
    return bad("pw_add_rms_norm: a residual output needs a residual");
  if (T == 0) return PW_OK;
  if (!d_x || !d_weight || !d_y || (y_type == PW_E4M3 && !d_scales))
    return bad("pw_add_rms_norm: null buffer");
  if (x_stride < 0 || residual_stride < 0 || residual_out_stride < 0 || y_stride < 0 ||
      (T > 1 && (y_stride < H || (d_residual_out && residual_out_stride < H))))
    return bad("pw_add_rms_norm: row strides are not negative, and outputs' at least H");
  // in place a row must lie where the row it replaces lies
  auto clash = [&](const void* out, int out_type, int64_t out_ld, const void* in, int in_type,
                   int64_t in_ld) {
    return out && out == in && (out_type != in_type || (T > 1 && out_ld != in_ld));
  };
  if (clash(d_y, y_type, y_stride, d_x, x_type, x_stride) ||
      clash(d_y, y_type, y_stride, d_residual, residual_type, residual_stride) ||
      clash(d_residual_out, residual_type, residual_out_stride, d_x, x_type, x_stride) ||
      clash(d_residual_out, residual_type, residual_out_stride, d_residual, residual_type,
            residual_stride) ||
      d_residual_out == d_y)
    return bad("pw_add_rms_norm: outputs in place have their input's type and stride, and two outputs "
               "two places");
  if (!aligned_to(d_x, type_bytes(x_type)) || !aligned_to(d_weight, type_bytes(weight_type)) ||
      !aligned_to(d_y, type_bytes(y_type)) ||
      (d_residual && !aligned_to(d_residual, type_bytes(residual_type))) ||
      (d_residual_out && !aligned_to(d_residual_out, type_bytes(residual_type))) ||
      (d_scales && !aligned_to(d_scales, 4)))
    return bad("pw_add_rms_norm: buffers must be aligned to their elements");
  int dev = 0, n_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return record_error(PW_ERR_CUDA, cudaGetErrorString(e));
  NormParams p{};
  p.x = d_x;
  p.res = d_residual;
  p.w = d_weight;
  p.res_out = d_residual_out;
  p.y = d_y;
  p.scales = d_scales;
  p.x_ld = x_stride;
  p.res_ld = residual_stride;
  p.res_out_ld = residual_out_stride;
  p.y_ld = y_stride;
  p.T = T;
  p.H = H;
  p.n_groups = (H + kGroup - 1) / kGroup;
  p.w_f32 = weight_type == PW_F32;
  p.eps = eps;
  p.inv_h = 1.0f / static_cast<float>(H);
  const int out = y_type == PW_BF16 ? kOutBf16 : scale_group == 0 ? kOutE4m3Row : kOutE4m3Group;
  const bool vec = H % 8 == 0 && vec_ok(d_x, x_stride, x_type) &&
                   vec_ok(d_residual, residual_stride, residual_type) &&
                   vec_ok(d_weight, 0, weight_type) &&
                   vec_ok(d_residual_out, residual_out_stride, residual_type) &&
                   vec_ok(d_y, y_stride, y_type);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  e = x_type == PW_F32 ? launch_x<float>(p, residual_type, out, vec, n_sm, s)
                       : launch_x<__nv_bfloat16>(p, residual_type, out, vec, n_sm, s);
  if (e != cudaSuccess) return record_error(PW_ERR_CUDA, cudaGetErrorString(e));
  return PW_OK;
}
