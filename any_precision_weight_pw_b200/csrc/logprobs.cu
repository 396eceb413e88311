// logprobs.cu -- pw_token_logprobs: log probabilities of given tokens, the
// entropy and the n best alternatives of a softmax over each row of logits.
//
// One pass over the logits.  With a running reference r (the largest logit
// seen so far) every thread keeps
//   s = sum exp(z - r),   u = sum exp(z - r) (z - r),
// rescaled by exp(r_old - r_new) when r grows (u gains s (r_old - r_new)
// first).  Over the row: log p_j = z_j - r - ln s, entropy = ln s - u / s; both
// of its terms are >= 0, so nothing cancels.  z - r is formed before the
// multiplication by log2 e, so large logits lose no digits.
//
// The n best come from the same pass.  Every thread also keeps its best
// vector: (largest logit, first such vector).  The n-th largest of these over
// the block's groups of 8 threads is a bound that at least n logits reach, and
// a logit reaching it can only lie with a thread whose best vector does: only
// those threads' logits (about n / 512 of the row) are read a second time.  The
// few logits that reach the bound are put in order by counting, for each, the
// larger ones.  Keys carry the index below the logit, so all keys differ and
// ties fall to the lower index.
//
// Few rows are split over a cluster; the blocks' sums and lists meet in the
// first block's shared memory in rank order, so results never depend on timing.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>

#include "pw_internal.h"

namespace pw {
namespace {

constexpr int kLpThreads = 512;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpMaxCluster = 8;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kFar = -200.0f;  // exp(-200) is zero in fp32: z - r stops here, so 0 * -inf never forms

struct LogprobParams {
  const void* z;
  int64_t ld;
  const int32_t* tokens;
  float* logprob;
  float* entropy;
  int32_t* top_idx;
  float* top_logprob;
  int V, n_top, n_split;  // n_split: blocks of the row's cluster
};

// 16 bytes of logits
template <typename T>
struct LogitVec;
template <>
struct LogitVec<float> {
  static constexpr int N = 4;
  static __device__ float one(const void* p, int64_t i) { return static_cast<const float*>(p)[i]; }
  static __device__ void widen(const uint4& q, float* v) {
    v[0] = __uint_as_float(q.x);
    v[1] = __uint_as_float(q.y);
    v[2] = __uint_as_float(q.z);
    v[3] = __uint_as_float(q.w);
  }
};
template <>
struct LogitVec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ float one(const void* p, int64_t i) {
    return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16);
  }
  static __device__ void widen(const uint4& q, float* v) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = __uint_as_float(w[k] << 16);
      v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
  }
};
template <>
struct LogitVec<__half> {
  static constexpr int N = 8;
  static __device__ float one(const void* p, int64_t i) {
    return __half2float(static_cast<const __half*>(p)[i]);
  }
  static __device__ void widen(const uint4& q, float* v) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __half2 h = *reinterpret_cast<const __half2*>(&w[k]);
      v[2 * k] = __low2float(h);
      v[2 * k + 1] = __high2float(h);
    }
  }
};

__device__ __forceinline__ uint4 load_stream(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// One special-function instruction for e^d as 2^(d log2 e).  Its error and the
// rounded product's, 2^-21 for the d that carry a softmax, stay in s and u: 6.2e-8
// relative error of the outputs against float64 at 4096 x 128000 fp32, 5.6e-8 for
// torch's exp in fp32.
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// two fp32 lanes, each correctly rounded
typedef unsigned long long f2;
__device__ __forceinline__ f2 pack2(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(f2 v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Keys order logits: larger first, then the lower index; 0 is below every key.
// Adding +0 makes -0 equal +0; a NaN of either sign is above +inf.
__device__ __forceinline__ int order_of(float z) {
  const int b = __float_as_int(__fadd_rn(z, 0.0f));
  return z != z ? 0x7fffffff : b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ unsigned long long make_key(int order, int idx) {
  return (static_cast<unsigned long long>(static_cast<uint32_t>(order) ^ 0x80000000u) << 32) |
         static_cast<uint32_t>(~idx);
}
__device__ __forceinline__ int key_index(unsigned long long k) {
  return static_cast<int>(~static_cast<uint32_t>(k));
}
__device__ __forceinline__ float key_logit(unsigned long long k) {
  const int o = static_cast<int>(static_cast<uint32_t>(k >> 32) ^ 0x80000000u);
  return __int_as_float(o ^ ((o >> 31) & 0x7fffffff));
}

constexpr int kGroups = kLpThreads / 8;  // groups of 8 threads
constexpr int kMaxCand = 1024;

__device__ __forceinline__ unsigned long long shfl_max(unsigned long long k, int j) {
  const unsigned long long o = __shfl_xor_sync(0xffffffffu, k, j);
  return k > o ? k : o;
}
// How many of keys[0..n) are larger (n even).
__device__ __forceinline__ int larger(const unsigned long long* keys, int n, unsigned long long k) {
  int r = 0;
#pragma unroll 4
  for (int i = 0; i < n; i += 2) {
    const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(keys + i);
    r += (o.x > k) + (o.y > k);
  }
  return r;
}

struct Sums {
  float r, s, u;
};
__device__ __forceinline__ Sums rescaled(const Sums& a, float r) {
  const float d = max_nan(a.r - r, kFar), f = ex2(d * kLog2e);
  return {r, a.s * f, fmaf(a.s, d, a.u) * f};
}
__device__ __forceinline__ void merge_lanes(Sums& a) {
  float r = a.r;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) r = max_nan(r, __shfl_xor_sync(0xffffffffu, r, o));
  a = rescaled(a, r);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a.s += __shfl_xor_sync(0xffffffffu, a.s, o);
    a.u += __shfl_xor_sync(0xffffffffu, a.u, o);
  }
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// the address in cluster block 0 of a shared-memory variable of this block
__device__ __forceinline__ uint32_t in_block0(const void* p) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;"
               : "=r"(r)
               : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))));
  return r;
}

// U: vectors a thread loads at once; B: blocks an SM.  Measured at 4096 rows of
// 128000: fp32 alone 296 us with 4 vectors and 2 blocks, 335 with 2 and 4;
// with alternatives (1024 rows) 132 and 115; bf16 210 us with 2 vectors and 2
// blocks, 170 with 1 and 4.
template <typename ZT, bool TOP, int U, int B>
__global__ void __launch_bounds__(kLpThreads, B) logprob_kernel(const LogprobParams p) {
  constexpr int N = LogitVec<ZT>::N;
  __shared__ Sums part[kLpWarps];
  __shared__ Sums slot_sums[kLpMaxCluster];
  __shared__ __align__(16) unsigned long long s_group[TOP ? kGroups : 2];  // groups' best, then lists
  __shared__ __align__(16) unsigned long long s_list[TOP ? kLpMaxCluster * 32 : 2];
  __shared__ __align__(16) unsigned long long s_cand[TOP ? kMaxCand : 2];
  __shared__ uint16_t s_thread[TOP ? kLpThreads : 1];
  __shared__ unsigned long long s_bound;
  __shared__ int s_threads, s_cands;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n_split = p.n_split;
  const int rank = n_split > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int64_t row = blockIdx.x / n_split;
  if (n_split > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  pdl_wait();

  // the row as head | 16-byte vectors | tail; this block's vectors are [v0, v1)
  const ZT* z = static_cast<const ZT*>(p.z) + row * p.ld;
  const int mis = static_cast<int>((reinterpret_cast<uintptr_t>(z) & 15) / sizeof(ZT));
  const int head = min(p.V, mis ? N - mis : 0);
  const int n_vec = (p.V - head) / N, tail0 = head + n_vec * N;
  const int per = (n_vec + n_split - 1) / n_split;
  const int v0 = min(n_vec, rank * per), v1 = min(n_vec, v0 + per);
  const uint4* zv = reinterpret_cast<const uint4*>(z + head);
  const bool has_head = rank == 0 && tid < head;
  const bool has_tail = rank == n_split - 1 && tid < p.V - tail0;
  float z_tok = 0.f;
  int tok = -1;
  if (p.tokens && rank == 0 && tid == 0) {
    tok = p.tokens[row];
    if (tok >= 0 && tok < p.V) z_tok = LogitVec<ZT>::one(z, tok);
  }

  Sums a = {-FLT_MAX, 0.f, 0.f};
  int best = INT32_MIN, best_at = 0;  // largest logit's order and where its vector starts
  auto absorb_one = [&](int i) {
    const float v = LogitVec<ZT>::one(z, i);
    a = rescaled(a, max_nan(a.r, v));
    const float d = max_nan(v - a.r, kFar), e = ex2(d * kLog2e);
    a.s += e;
    a.u = fmaf(e, d, a.u);
    if (TOP) {
      const int o = order_of(v);
      if (o > best) best = o, best_at = i;
    }
  };
  if (has_head) absorb_one(tid);
  // even and odd logits of a vector sum apart, two at a time
  f2 s2 = pack2(a.s, 0.f), u2 = pack2(a.u, 0.f);
  for (int v = v0 + tid; v < v1; v += U * kLpThreads) {
    uint4 q[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int i = v + k * kLpThreads;
      if (i < v1) q[k] = load_stream(zv + i);
    }
    float x[U][N], mx = a.r;
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int i = v + k * kLpThreads;
      if (i < v1) {
        LogitVec<ZT>::widen(q[k], x[k]);
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j) x[k][j] = __int_as_float(0xff800000);
      }
      float m = x[k][0];
#pragma unroll
      for (int j = 1; j < N; ++j) m = max_nan(m, x[k][j]);
      mx = max_nan(mx, m);
      if (TOP) {
        const int o = order_of(m);
        if (i < v1 && o > best) best = o, best_at = head + i * N;
      }
    }
    {
      const float d = max_nan(a.r - mx, kFar), f = ex2(d * kLog2e);
      const f2 f_2 = pack2(f, f);
      u2 = mul2(fma2(s2, pack2(d, d), u2), f_2);
      s2 = mul2(s2, f_2);
      a.r = mx;
    }
    const f2 minus = pack2(-mx, -mx), scale = pack2(kLog2e, kLog2e);
#pragma unroll
    for (int k = 0; k < U; ++k)
#pragma unroll
      for (int j = 0; j < N; j += 2) {
        float d0, d1, t0, t1;
        unpack2(add2(pack2(x[k][j], x[k][j + 1]), minus), d0, d1);
        const f2 d = pack2(max_nan(d0, kFar), max_nan(d1, kFar));
        unpack2(mul2(d, scale), t0, t1);
        const f2 e = pack2(ex2(t0), ex2(t1));
        s2 = add2(s2, e);
        u2 = fma2(e, d, u2);
      }
  }
  {
    float lo, hi;
    unpack2(s2, lo, hi);
    a.s = lo + hi;
    unpack2(u2, lo, hi);
    a.u = lo + hi;
  }
  if (has_tail) absorb_one(tail0 + tid);

  merge_lanes(a);
  if (lane == 0) part[warp] = a;
  unsigned long long mine = 0;  // warp 0: lane i holds the block's i-th best
  if (TOP) {
    const int n = p.n_top;
    const unsigned long long key = best == INT32_MIN ? 0ull : make_key(best, best_at);
    const unsigned long long gk = shfl_max(shfl_max(shfl_max(key, 1), 2), 4);
    if ((lane & 7) == 0) s_group[tid >> 3] = gk;
    if (tid < 32) s_list[tid] = 0;
    if (tid == 0) s_threads = s_cands = 0, s_bound = 0;
    __syncthreads();
    // the n-th best group's key (0 with fewer groups in use: every logit counts)
    if (tid < kGroups && s_group[tid] != 0 && larger(s_group, kGroups, s_group[tid]) == n - 1)
      s_bound = s_group[tid];
    __syncthreads();
    const unsigned long long bound = s_bound;
    // A logit reaches the bound if it is larger, or equal and not behind the
    // bound's vector.
    const uint32_t last = bound ? ~(static_cast<uint32_t>(key_index(bound)) + N - 1) : 0u;
    const unsigned long long reach = (bound & 0xffffffff00000000ull) | last;
    if (key != 0 && key >= bound) s_thread[atomicAdd(&s_threads, 1)] = static_cast<uint16_t>(tid);
    __syncthreads();
    // visit(key) for every logit of the listed threads, a warp a thread
    const int n_threads = s_threads;
    auto scan = [&](auto visit) {
      for (int j = warp; j < n_threads; j += kLpWarps) {
        const int owner = s_thread[j];
        if (lane == 0 && rank == 0 && owner < head)
          visit(make_key(order_of(LogitVec<ZT>::one(z, owner)), owner));
        if (lane == 1 && rank == n_split - 1 && owner < p.V - tail0)
          visit(make_key(order_of(LogitVec<ZT>::one(z, tail0 + owner)), tail0 + owner));
        for (int64_t i = v0 + owner + static_cast<int64_t>(lane) * kLpThreads; i < v1;
             i += 32 * kLpThreads) {
          float x[N];
          LogitVec<ZT>::widen(zv[i], x);
#pragma unroll
          for (int e = 0; e < N; ++e)
            visit(make_key(order_of(x[e]), head + static_cast<int>(i) * N + e));
        }
      }
    };
    scan([&](unsigned long long k) {
      if (k < reach) return;
      const int at = atomicAdd(&s_cands, 1);
      if (at < kMaxCand) s_cand[at] = k;
    });
    __syncthreads();
    const int n_cand = s_cands;
    if (n_cand <= kMaxCand) {  // the same order whatever order they came in
      if (tid == 0 && (n_cand & 1)) s_cand[n_cand] = 0;  // kMaxCand is even
      __syncthreads();
      for (int i = tid; i < n_cand; i += kLpThreads) {
        const int r = larger(s_cand, (n_cand + 1) & ~1, s_cand[i]);
        if (r < n) s_list[r] = s_cand[i];
      }
    } else {  // many logits tie: one at a time
      unsigned long long below = ~0ull;
      for (int j = 0; j < n; ++j) {
        unsigned long long top = 0;
        scan([&](unsigned long long k) {
          if (k < below && k > top) top = k;
        });
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = shfl_max(top, o);
        if (lane == 0) s_group[warp] = top;
        __syncthreads();
        below = 0;
        for (int w = 0; w < kLpWarps; ++w) below = s_group[w] > below ? s_group[w] : below;
        if (tid == 0) s_list[j] = below;
        __syncthreads();
      }
    }
    __syncthreads();
    mine = s_list[lane];
  } else {
    __syncthreads();
  }
  if (warp == 0) {
    a = lane < kLpWarps ? part[lane] : Sums{-FLT_MAX, 0.f, 0.f};
    merge_lanes(a);
  }

  if (n_split > 1) {  // to the first block, which joins them in rank order
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (warp == 0) {
      if (lane == 0) {
        const uint32_t d = in_block0(&slot_sums[rank]);
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(d), "f"(a.r) : "memory");
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(d + 4), "f"(a.s) : "memory");
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(d + 8), "f"(a.u) : "memory");
      }
      if (TOP) {
        const uint32_t d = in_block0(&s_list[rank * 32 + lane]);
        asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(d), "l"(mine) : "memory");
      }
    }
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (rank != 0) return;
    if (TOP) {
      if (tid < 32) s_group[tid] = 0;
      __syncthreads();
      if (tid < 32 * n_split && s_list[tid] != 0) {
        const int r = larger(s_list, 32 * n_split, s_list[tid]);
        if (r < p.n_top) s_group[r] = s_list[tid];
      }
      __syncthreads();
      mine = s_group[lane];
    }
    if (warp == 0) {
      a = lane < n_split ? slot_sums[lane] : Sums{-FLT_MAX, 0.f, 0.f};
      merge_lanes(a);
    }
  }
  if (warp != 0) return;
  const bool none = a.s == 0.f;  // every logit -inf
  const float ln_s = logf(a.s);
  auto logprob = [&](float v) {
    return v == __int_as_float(0xff800000) ? v : (v - a.r) - ln_s;
  };
  if (lane == 0) {
    if (p.entropy) p.entropy[row] = none ? 0.f : ln_s - a.u / a.s;
    if (p.tokens)
      p.logprob[row] = tok == -1                 ? 0.f
                       : tok < 0 || tok >= p.V ? __int_as_float(0x7fffffff)
                                               : logprob(z_tok);
  }
  if (TOP && lane < p.n_top) {
    p.top_idx[row * p.n_top + lane] = key_index(mine);
    p.top_logprob[row * p.n_top + lane] = logprob(key_logit(mine));
  }
}

template <typename ZT, bool TOP>
cudaError_t launch_logprobs(LogprobParams p, int T, int n_sm, cudaStream_t s) {
  constexpr int N = LogitVec<ZT>::N, B = N == 4 && !TOP ? 2 : 4, U = B == 2 ? 4 : 8 / N;
  // rows are split while the blocks fill the GPU less than twice over and each
  // keeps a vector for every thread (64 rows of 128009 bf16 with alternatives:
  // 11.0 us in 4 parts, 18.0 in 8)
  int n_split = 1;
  while (n_split < kLpMaxCluster && static_cast<int64_t>(T) * n_split * 2 <= 2 * n_sm &&
         p.V >= n_split * 2 * kLpThreads * N)
    n_split *= 2;
  p.n_split = n_split;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(T) * static_cast<unsigned>(n_split));
  cfg.blockDim = dim3(kLpThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(n_split);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, logprob_kernel<ZT, TOP, U, B>, p);
}

template <typename ZT>
cudaError_t launch_type(const LogprobParams& p, int T, int n_sm, cudaStream_t s) {
  return p.n_top > 0 ? launch_logprobs<ZT, true>(p, T, n_sm, s)
                     : launch_logprobs<ZT, false>(p, T, n_sm, s);
}

}  // namespace
}  // namespace pw

extern "C" pw_status_t pw_token_logprobs(const void* d_logits, int32_t logits_type, int64_t stride,
                                         int32_t T, int32_t V, const int32_t* d_tokens,
                                         int32_t n_top, float* d_logprob, float* d_entropy,
                                         int32_t* d_top_idx, float* d_top_logprob,
                                         pw_stream_t stream) {
  using namespace pw;
  auto bad = [](const char* msg) { return record_error(PW_ERR_INVALID_ARG, msg); };
  if (T < 0 || V < 1) return bad("pw_token_logprobs: need T >= 0 and V >= 1");
  if (logits_type != PW_F32 && logits_type != PW_BF16 && logits_type != PW_F16)
    return bad("pw_token_logprobs: logits are PW_F32, PW_BF16 or PW_F16");
  if (n_top < 0 || n_top > PW_MAX_TOP_LOGPROBS || n_top > V)
    return bad("pw_token_logprobs: need 0 <= n_top <= min(V, 32)");
  if (stride < 0) return bad("pw_token_logprobs: the row stride is not negative");
  if (T == 0) return PW_OK;
  if (!d_logits || (d_tokens == nullptr) != (d_logprob == nullptr) ||
      (n_top > 0 && (!d_top_idx || !d_top_logprob)))
    return bad("pw_token_logprobs: null buffer (tokens and logprob go together)");
  const uintptr_t size = logits_type == PW_F32 ? 4 : 2;
  const uintptr_t words = reinterpret_cast<uintptr_t>(d_tokens) | reinterpret_cast<uintptr_t>(d_logprob) |
                          reinterpret_cast<uintptr_t>(d_entropy) |
                          reinterpret_cast<uintptr_t>(d_top_idx) |
                          reinterpret_cast<uintptr_t>(d_top_logprob);
  if (reinterpret_cast<uintptr_t>(d_logits) % size || words % 4)
    return bad("pw_token_logprobs: buffers must be aligned to their elements");
  int dev = 0, n_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return record_error(PW_ERR_CUDA, cudaGetErrorString(e));
  LogprobParams p{};
  p.z = d_logits;
  p.ld = stride;
  p.tokens = d_tokens;
  p.logprob = d_logprob;
  p.entropy = d_entropy;
  p.top_idx = d_top_idx;
  p.top_logprob = d_top_logprob;
  p.V = V;
  p.n_top = n_top;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  e = logits_type == PW_F32    ? launch_type<float>(p, T, n_sm, s)
      : logits_type == PW_BF16 ? launch_type<__nv_bfloat16>(p, T, n_sm, s)
                               : launch_type<__half>(p, T, n_sm, s);
  if (e != cudaSuccess) return record_error(PW_ERR_CUDA, cudaGetErrorString(e));
  return PW_OK;
}
