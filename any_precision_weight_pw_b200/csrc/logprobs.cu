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
// the block is a bound that at least n logits reach, and a logit reaching it
// can only lie with one of the n threads whose best vector does: only those
// n threads' logits (n / 512 of the row) are read a second time.  Keys carry
// the index below the logit, so all keys differ, ties fall to the lower index
// and a row of equal logits costs no more than another.
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
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
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

// 32 keys over the lanes, largest in lane 0 (bitonic).
__device__ __forceinline__ unsigned long long exchange(unsigned long long k, int j, bool keep_max) {
  const unsigned long long o = __shfl_xor_sync(0xffffffffu, k, j);
  return (k > o) == keep_max ? k : o;
}
__device__ __forceinline__ unsigned long long sort32(unsigned long long k) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int j = size >> 1; j > 0; j >>= 1)
      k = exchange(k, j, ((lane & j) == 0) == ((lane & size) == 0));
  return k;
}
// the 32 largest of two sorted lists, sorted
__device__ __forceinline__ unsigned long long merge32(unsigned long long a, unsigned long long b) {
  const int lane = threadIdx.x & 31;
  const unsigned long long o = __shfl_xor_sync(0xffffffffu, b, 31);  // b reversed
  unsigned long long k = a > o ? a : o;
#pragma unroll
  for (int j = 16; j > 0; j >>= 1) k = exchange(k, j, (lane & j) == 0);
  return k;
}
// Merges the sorted lists of warps 0..n-1 (n a power of two) into warp 0's;
// list: [n][32] shared.  Ends with a barrier; list[0..31] holds the result.
__device__ __forceinline__ unsigned long long merge_warps(unsigned long long k, int n,
                                                          unsigned long long* list) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (warp < n) list[warp * 32 + lane] = k;
  for (int step = 1; step < n; step <<= 1) {
    __syncthreads();
    if (warp < n && warp % (2 * step) == 0) {
      k = merge32(k, list[(warp + step) * 32 + lane]);
      list[warp * 32 + lane] = k;
    }
  }
  __syncthreads();
  return k;
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

template <typename ZT, bool TOP, int U>
__global__ void __launch_bounds__(kLpThreads) logprob_kernel(const LogprobParams p) {
  constexpr int N = LogitVec<ZT>::N;
  __shared__ Sums part[kLpWarps];
  __shared__ Sums slot_sums[kLpMaxCluster];
  __shared__ unsigned long long list[TOP ? kLpWarps * 32 : 1];
  __shared__ unsigned long long slot_keys[TOP ? kLpMaxCluster * 32 : 1];
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
    a = rescaled(a, mx);
#pragma unroll
    for (int k = 0; k < U; ++k)
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float d = max_nan(x[k][j] - mx, kFar), e = ex2(d * kLog2e);
        a.s += e;
        a.u = fmaf(e, d, a.u);
      }
  }
  if (has_tail) absorb_one(tail0 + tid);

  merge_lanes(a);
  if (lane == 0) part[warp] = a;
  unsigned long long mine = 0;  // warp 0: lane i holds the block's i-th best
  if (TOP) {
    const int n = p.n_top;
    merge_warps(sort32(best == INT32_MIN ? 0ull : make_key(best, best_at)), kLpWarps, list);
    const unsigned long long bound = list[n - 1];
    // A logit reaches the bound if it is larger, or equal and not behind the
    // bound's vector.  (A block with fewer than n threads in use: bound 0.)
    const uint32_t last = bound ? static_cast<uint32_t>(~(key_index(bound) + N - 1)) : 0u;
    const unsigned long long reach = (bound & 0xffffffff00000000ull) | last;
    for (int j = warp; j < n; j += kLpWarps) {
      const unsigned long long key = list[j];
      if (key == 0) break;
      // the thread whose best vector this is
      const int at = key_index(key);
      const int owner = at < head     ? at
                        : at >= tail0 ? at - tail0
                                      : ((at - head) / N - v0) % kLpThreads;
      auto offer = [&](unsigned long long c) {  // one key a lane, 0 for none
        if (c < reach) c = 0;
        if (__any_sync(0xffffffffu, c > __shfl_sync(0xffffffffu, mine, n - 1)))
          mine = merge32(mine, sort32(c));
      };
      unsigned long long c = 0;
      if (lane == 0 && rank == 0 && owner < head)
        c = make_key(order_of(LogitVec<ZT>::one(z, owner)), owner);
      if (lane == 1 && rank == n_split - 1 && owner < p.V - tail0)
        c = make_key(order_of(LogitVec<ZT>::one(z, tail0 + owner)), tail0 + owner);
      offer(c);
      for (int b = v0 + owner; b < v1; b += 32 * kLpThreads) {
        const int64_t i = b + static_cast<int64_t>(lane) * kLpThreads;
        float x[N];
        if (i < v1) {
          LogitVec<ZT>::widen(zv[i], x);
        }
#pragma unroll
        for (int e = 0; e < N; ++e)
          offer(i < v1 ? make_key(order_of(x[e]), head + static_cast<int>(i) * N + e) : 0ull);
      }
    }
    __syncthreads();  // every warp has read the bound and its threads
    mine = merge_warps(mine, kLpWarps, list);
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
        const uint32_t d = in_block0(&slot_keys[rank * 32 + lane]);
        asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(d), "l"(mine) : "memory");
      }
    }
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (rank != 0) return;
    if (TOP) mine = merge_warps(warp < n_split ? slot_keys[warp * 32 + lane] : 0ull, n_split, list);
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
  constexpr int N = LogitVec<ZT>::N, U = 16 / N * 1;
  // rows are split while the blocks do not fill the GPU and each keeps a
  // vector for every thread
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
  return cudaLaunchKernelEx(&cfg, logprob_kernel<ZT, TOP, U>, p);
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
