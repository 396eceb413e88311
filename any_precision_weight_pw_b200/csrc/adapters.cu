// adapters.cu -- pw_adapters: low-rank adapters of many requests beside one
// shared projection, y_t = base_t + scale_a * B_a (A_a x_t), a = ids[t].
//
// One launch, no workspace.  A cluster of 8 blocks takes R tokens and keeps
// everything between its two products on chip:
//   order    the tokens of a window of 256 are taken in the order of their
//            adapters where they are mixed, so tokens that share an adapter
//            meet in one cluster, and cut into pieces of at most 16 tokens of
//            one adapter (the rows of an MMA tile);
//   shrink   v = A_a x: block c of the cluster takes an eighth of the columns,
//            its warps split that again; the partial sums meet over distributed
//            shared memory, in a fixed order;
//   expand   y = base + B_a (scale v): block c takes an eighth of the rows.
// Both products run on mma.sync m16n8k16 (bf16, fp32 accumulation) straight
// from global memory: the contraction index may be permuted freely as long as
// both operands agree, so each lane loads 16 (shrink) or 8 (expand) contiguous
// bytes of a row and uses them as its fragments of two or one MMA steps.
// At ranks up to 64 the operator needs at most about 50 operations a byte, a
// fifth of what this GPU's tensor cores could do per byte of its memory, so
// the wide tcgen05 tiles, which would need x and B staged in shared memory,
// have nothing to win here; what counts is bytes in flight.
//
// Precision.  v is split into bf16 terms (v = hi + mid + lo, 24 bits; two
// terms, 16 bits, when y is bf16 and rounds to 8), each multiplied with B
// exactly; sums are fp32.
#include <cuda_bf16.h>

#include <cmath>
#include <mutex>

#include "pw_internal.h"

namespace pw {
namespace {

constexpr int kAdThreads = 256;
constexpr int kAdWarps = kAdThreads / 32;
constexpr int kAdCluster = 8;
constexpr int kWindow = 256;   // tokens ordered together
constexpr int kMaxRows = 64;   // tokens of a cluster
constexpr int kMaxDevices = 64;

struct AdapterParams {
  const uint16_t* x;
  const uint16_t* a;
  const uint16_t* b;
  const int32_t* ids;
  const int32_t* ranks;
  const float* scale;
  const void* base;
  void* y;
  int64_t x_ld, base_ld, y_ld;
  int n, r_max, T, cols, rows;
  int R;          // tokens of a cluster (a power of two, at most 16 * MT)
  int v_ld;       // bf16 elements between the rows of v in shared memory
  int vec_x;      // 16-byte loads of x and A are legal
  int vec_b;      // 8-byte loads of B are legal
  int vec_y;      // 16-byte (fp32) or 8-byte (bf16) accesses of base and y are legal
  int y_f32;
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ uint32_t in_block(uint32_t addr, int rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void put4(uint32_t addr, const float4& v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x), "f"(v.y),
               "f"(v.z), "f"(v.w)
               : "memory");
}

__device__ __forceinline__ void mma16816(float* c, uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// `count` (at most 8) bf16 from p on, zero past them, as 16 bytes
__device__ __forceinline__ uint4 load8(const uint16_t* p, int count, bool vec) {
  uint4 v = make_uint4(0, 0, 0, 0);
  if (count <= 0) return v;
  if (vec) return __ldg(reinterpret_cast<const uint4*>(p));
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = i < count ? __ldg(p + i) : 0u;
  return make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
}
__device__ __forceinline__ uint2 load4(const uint16_t* p, int count, bool vec) {
  uint2 v = make_uint2(0, 0);
  if (count <= 0) return v;
  if (vec && count >= 4) return __ldg(reinterpret_cast<const uint2*>(p));
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = i < count ? __ldg(p + i) : 0u;
  return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

__device__ __forceinline__ float bf16_value(uint16_t b) {
  return __uint_as_float(static_cast<uint32_t>(b) << 16);
}
__device__ __forceinline__ uint16_t bf16_bits(float v) {
  return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

struct Piece {
  int start, len, adapter, rank;  // rank 0: nothing to add (no adapter)
};

// MT: pieces worked on at once (the warps split into MT groups); NT: 8-wide
// rank tiles of a shrink step (rank chunks of 8 * NT).
template <int MT, int NT>
__global__ void __launch_bounds__(kAdThreads) adapter_kernel(const AdapterParams p) {
  constexpr int KW = kAdWarps / MT;       // warps sharing a piece
  constexpr int kChunk = 8 * NT;          // ranks of a shrink step
  constexpr int kTile = 16 * kChunk;      // partial sums of a piece and step
  constexpr bool kTwoStep = MT > 1;       // partial sums: reduce-scatter + all-gather
  // slots: one step, every block gets every block's sums (two buffers in turn);
  // two steps, a block gets its eighth of them
  constexpr int kSlot = kTwoStep ? MT * kTile / kAdCluster : kTile;
  extern __shared__ __align__(16) uint8_t smem[];
  float* red = reinterpret_cast<float*>(smem);             // [8 warps][16][kChunk]
  float* slots = red + kAdWarps * kTile;                   // [2 or 1][8 blocks][kSlot]
  uint16_t* vt = reinterpret_cast<uint16_t*>(slots + (kTwoStep ? 1 : 2) * kAdCluster * kSlot);
  __shared__ __align__(16) int s_key[kWindow];
  __shared__ int s_tok[kMaxRows], s_id[kMaxRows];
  __shared__ Piece s_piece[kMaxRows];
  __shared__ int s_np;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, q = lane & 3;
  const int rank = static_cast<int>(cluster_rank());
  const int cl = blockIdx.x / kAdCluster;
  const int per_window = kWindow / p.R;
  const int t0 = cl / per_window * kWindow;               // the window's first token
  const int n_win = min(kWindow, p.T - t0);
  const int first = cl % per_window * p.R;                // the cluster's first position
  const int n_rows = min(p.R, n_win - first);             // >= 1 by the grid
  cluster_arrive();  // the other blocks' shared memory is live once all have arrived
  pdl_wait();

  // ---- order: this cluster's tokens and its pieces ------------------------
  if (p.R == 1) {
    if (tid == 0) {
      const int id = p.ids[t0 + first];
      s_tok[0] = t0 + first;
      s_id[0] = id >= 0 && id < p.n ? id : -1;
    }
  } else {
    int id = -1;
    if (tid < n_win) {
      id = p.ids[t0 + tid];
      if (id < 0 || id >= p.n) id = -1;
    }
    // id 0..n-1, none = 2^22 - 1; the position in the low 8 bits
    const int key = ((id < 0 ? PW_MAX_ADAPTERS : id) << 8) | tid;
    s_key[tid] = tid < n_win ? key : INT32_MAX;
    __syncthreads();
    const bool change = tid > 0 && tid < n_win && (s_key[tid - 1] >> 8) != (key >> 8);
    const int runs = 1 + __syncthreads_count(change);
    int pos = tid;
    if (runs * 16 > n_win) {  // mixed: position = number of smaller keys
      pos = 0;
      for (int i = 0; i < n_win; i += 4) {
        const int4 k4 = *reinterpret_cast<const int4*>(s_key + i);
        pos += (k4.x < key) + (k4.y < key) + (k4.z < key) + (k4.w < key);
      }
    }
    if (tid < n_win && pos >= first && pos < first + n_rows) {
      s_tok[pos - first] = t0 + tid;
      s_id[pos - first] = id;
    }
  }
  __syncthreads();
  if (warp == 0) {
    // a piece starts where the adapter changes and at every 16th token of a run
    uint64_t changes = 0;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int i = lane + 32 * half;
      const bool c = i < n_rows && (i == 0 || s_id[i] != s_id[i - 1]);
      changes |= static_cast<uint64_t>(__ballot_sync(0xffffffffu, c)) << (32 * half);
    }
    uint64_t starts = 0;
    bool is_start[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int i = lane + 32 * half;
      const uint64_t upto = changes & (~0ull >> (63 - i));
      is_start[half] = i < n_rows && (i - (63 - __clzll(upto))) % 16 == 0;
      starts |= static_cast<uint64_t>(__ballot_sync(0xffffffffu, is_start[half])) << (32 * half);
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int i = lane + 32 * half;
      if (!is_start[half]) continue;
      const uint64_t above = i == 63 ? 0ull : starts & (~0ull << (i + 1));
      const int id = s_id[i];
      int r = 0;
      if (id >= 0) r = p.ranks ? min(max(p.ranks[id], 0), p.r_max) : p.r_max;
      s_piece[__popcll(starts & ((1ull << i) - 1))] = {
          i, (above ? __ffsll(above) - 1 : n_rows) - i, id, r};
    }
    if (lane == 0) s_np = __popcll(starts);
  }
  __syncthreads();
  const int n_pieces = s_np;
  const int mp = warp % MT, kw = warp / MT;  // piece and share of this warp

  // this block's columns (shrink, in 32s) and rows (expand, in 32s)
  const int kb_all = (p.cols + 31) / 32, ob_all = (p.rows + 31) / 32;
  const int kb0 = rank * kb_all / kAdCluster, kb1 = (rank + 1) * kb_all / kAdCluster;
  const int ob0 = rank * ob_all / kAdCluster, ob1 = (rank + 1) * ob_all / kAdCluster;
  const int v_plane = 16 * MT * p.v_ld;      // one bf16 term of v
  const int n_terms = p.y_f32 ? 3 : 2;
  cluster_wait();

  int step = 0;  // exchange steps done: the one-step slots alternate
  for (int p0 = 0; p0 < n_pieces; p0 += MT) {
    Piece pc = {0, 0, -1, 0};
    if (p0 + mp < n_pieces) pc = s_piece[p0 + mp];
    int r_all = 0;  // largest rank of this pass: the same in all blocks
    for (int i = p0; i < min(n_pieces, p0 + MT); ++i) r_all = max(r_all, s_piece[i].rank);

    // ---- shrink ------------------------------------------------------------
    for (int r0 = 0; r0 < r_all; r0 += kChunk, ++step) {
      float acc[NT][4];
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
      const int nr = min(kChunk, pc.rank - r0);  // ranks of this piece here (may be <= 0)
      if (nr > 0) {
        const uint16_t* x0 = p.x + (g < pc.len ? s_tok[pc.start + g] : 0) * p.x_ld;
        const uint16_t* x1 = p.x + (g + 8 < pc.len ? s_tok[pc.start + g + 8] : 0) * p.x_ld;
        const uint16_t* ar = p.a + (static_cast<int64_t>(pc.adapter) * p.r_max + r0 + g) * p.cols;
#pragma unroll 2
        for (int kb = kb0 + kw; kb < kb1; kb += KW) {
          const int c = kb * 32 + q * 8;
          const int left = p.cols - c;
          const uint4 xa = load8(x0 + c, g < pc.len ? left : 0, p.vec_x);
          const uint4 xb = load8(x1 + c, g + 8 < pc.len ? left : 0, p.vec_x);
          uint4 w[NT];
#pragma unroll
          for (int j = 0; j < NT; ++j)
            w[j] = load8(ar + static_cast<int64_t>(8 * j) * p.cols + c, 8 * j + g < nr ? left : 0,
                         p.vec_x);
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            mma16816(acc[j], xa.x, xb.x, xa.y, xb.y, w[j].x, w[j].y);
            mma16816(acc[j], xa.z, xb.z, xa.w, xb.w, w[j].z, w[j].w);
          }
        }
      }
      float* mine = red + warp * kTile;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        *reinterpret_cast<float2*>(mine + g * kChunk + 8 * j + 2 * q) =
            make_float2(acc[j][0], acc[j][1]);
        *reinterpret_cast<float2*>(mine + (g + 8) * kChunk + 8 * j + 2 * q) =
            make_float2(acc[j][2], acc[j][3]);
      }
      __syncthreads();
      // sums over this block's warps, to the blocks that need them
      for (int e = tid * 4; e < MT * kTile; e += kAdThreads * 4) {
        const int m = e / kTile, i = e % kTile;
        float4 s = *reinterpret_cast<const float4*>(red + m * kTile + i);
#pragma unroll
        for (int k = 1; k < KW; ++k) {
          const float4 o = *reinterpret_cast<const float4*>(red + (k * MT + m) * kTile + i);
          s.x += o.x, s.y += o.y, s.z += o.z, s.w += o.w;
        }
        if (kTwoStep) {
          put4(in_block(smem_u32(slots + rank * kSlot + e % kSlot), e / kSlot), s);
        } else {
          const uint32_t d = smem_u32(slots + ((step & 1) * kAdCluster + rank) * kSlot + e);
#pragma unroll
          for (int c = 0; c < kAdCluster; ++c) put4(in_block(d, c), s);
        }
      }
      cluster_arrive();
      cluster_wait();
      // sums over the blocks; scale v and split it into bf16 terms
      const float* from = slots + (kTwoStep ? 0 : (step & 1) * kAdCluster * kSlot);
      for (int e = tid * 2; e < kSlot; e += kAdThreads * 2) {
        float2 s = make_float2(0.f, 0.f);
#pragma unroll
        for (int c = 0; c < kAdCluster; ++c) {
          const float2 o = *reinterpret_cast<const float2*>(from + c * kSlot + e);
          s.x += o.x, s.y += o.y;
        }
        const int f = kTwoStep ? rank * kSlot + e : e;  // [MT][16][kChunk]
        const int m = f / kTile, row = f % kTile / kChunk, k = r0 + f % kChunk;
        if (k >= p.v_ld || p0 + m >= n_pieces) continue;
        const int id = s_piece[p0 + m].adapter;
        const float sc = id >= 0 && p.scale ? p.scale[id] : 1.f;
        float v[2] = {s.x * sc, s.y * sc};
        const uint32_t d = smem_u32(vt + (m * 16 + row) * p.v_ld + k);
        for (int t = 0; t < n_terms; ++t) {
          uint16_t h[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            h[i] = bf16_bits(v[i]);
            const float hv = bf16_value(h[i]);
            v[i] = fabsf(hv) < INFINITY ? v[i] - hv : 0.f;  // infinities and NaN are whole in one term
          }
          const uint32_t w = h[0] | static_cast<uint32_t>(h[1]) << 16;
          if (kTwoStep) {
#pragma unroll
            for (int c = 0; c < kAdCluster; ++c)
              asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(
                               in_block(d + static_cast<uint32_t>(t * v_plane * 2), c)),
                           "r"(w)
                           : "memory");
          } else {
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(d + static_cast<uint32_t>(t * v_plane * 2)),
                         "r"(w)
                         : "memory");
          }
        }
      }
      if (kTwoStep) {
        cluster_arrive();
        cluster_wait();
      } else {
        __syncthreads();
      }
    }

    // ---- expand --------------------------------------------------------------
    if (pc.len > 0 && (pc.rank > 0 || p.base != p.y)) {
      const bool on0 = g < pc.len, on1 = g + 8 < pc.len;
      const int64_t row0 = on0 ? s_tok[pc.start + g] : 0, row1 = on1 ? s_tok[pc.start + g + 8] : 0;
      const uint16_t* vrow = vt + (mp * 16 + g) * p.v_ld + 4 * q;
      const uint16_t* br = p.b + static_cast<int64_t>(pc.adapter) * p.rows * p.r_max;
      // n index g of MMA tile j is row o + 16 (j / 2) + 4 (g / 2) + 2 (j % 2) + g % 2:
      // a lane then holds rows 4q..4q+3 of each half of the 32
      const int og = 4 * (g >> 1) + (g & 1);
      for (int ob = ob0 + kw; ob < ob1; ob += KW) {
        const int o = ob * 32;
        float acc[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
        float add[2][2][4];  // [token half][row half]: base
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const int c = o + 16 * w + 4 * q;
            const int64_t at = (h ? row1 : row0) * p.base_ld + c;
            float* d = add[h][w];
            d[0] = d[1] = d[2] = d[3] = 0.f;
            if (!p.base || !(h ? on1 : on0) || c >= p.rows) continue;
            if (p.y_f32) {
              const float* src = static_cast<const float*>(p.base) + at;
              if (p.vec_y) {
                const float4 v = *reinterpret_cast<const float4*>(src);
                d[0] = v.x, d[1] = v.y, d[2] = v.z, d[3] = v.w;
              } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (c + i < p.rows) d[i] = src[i];
              }
            } else {
              const uint16_t* src = static_cast<const uint16_t*>(p.base) + at;
              if (p.vec_y) {
                const uint2 v = *reinterpret_cast<const uint2*>(src);
                d[0] = __uint_as_float(v.x << 16), d[1] = __uint_as_float(v.x & 0xffff0000u);
                d[2] = __uint_as_float(v.y << 16), d[3] = __uint_as_float(v.y & 0xffff0000u);
              } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (c + i < p.rows) d[i] = bf16_value(src[i]);
              }
            }
          }
#pragma unroll 2
        for (int k0 = 0; k0 < pc.rank; k0 += 16) {
          uint2 w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int ro = o + 16 * (j >> 1) + 2 * (j & 1) + og;
            w[j] = load4(br + static_cast<int64_t>(ro) * p.r_max + k0 + 4 * q,
                         ro < p.rows ? pc.rank - k0 - 4 * q : 0, p.vec_b);
          }
          for (int t = 0; t < n_terms; ++t) {
            const uint16_t* vp = vrow + t * v_plane + k0;
            const uint2 lo = *reinterpret_cast<const uint2*>(vp);
            const uint2 hi = *reinterpret_cast<const uint2*>(vp + 8 * p.v_ld);
#pragma unroll
            for (int j = 0; j < 4; ++j) mma16816(acc[j], lo.x, hi.x, lo.y, hi.y, w[j].x, w[j].y);
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const int c = o + 16 * w + 4 * q;
            if (!(h ? on1 : on0) || c >= p.rows) continue;
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = add[h][w][i] + acc[2 * w + (i >> 1)][2 * h + (i & 1)];
            const int64_t at = (h ? row1 : row0) * p.y_ld + c;
            if (p.y_f32) {
              float* dst = static_cast<float*>(p.y) + at;
              if (p.vec_y) {
                *reinterpret_cast<float4*>(dst) = make_float4(v[0], v[1], v[2], v[3]);
              } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (c + i < p.rows) dst[i] = v[i];
              }
            } else {
              uint16_t* dst = static_cast<uint16_t*>(p.y) + at;
              if (p.vec_y) {
                *reinterpret_cast<uint2*>(dst) =
                    make_uint2(bf16_bits(v[0]) | static_cast<uint32_t>(bf16_bits(v[1])) << 16,
                               bf16_bits(v[2]) | static_cast<uint32_t>(bf16_bits(v[3])) << 16);
              } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (c + i < p.rows) dst[i] = bf16_bits(v[i]);
              }
            }
          }
      }
    }
  }
}

template <int MT, int NT>
cudaError_t launch_shape(const AdapterParams& p, cudaStream_t s) {
  constexpr int kTile = 16 * 8 * NT;
  constexpr size_t kSums =
      sizeof(float) * (kAdWarps * kTile + (MT > 1 ? MT * kTile : 2 * kAdCluster * kTile));
  constexpr int kMaxLd = PW_MAX_ADAPTER_RANK + 16;
  const size_t smem = kSums + sizeof(uint16_t) * (p.y_f32 ? 3 : 2) * 16 * MT * p.v_ld;
  static std::mutex mu;
  static bool attr_set[kMaxDevices] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!attr_set[dev]) {
      e = cudaFuncSetAttribute(adapter_kernel<MT, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(kSums + sizeof(uint16_t) * 3 * 16 * MT * kMaxLd));
      if (e != cudaSuccess) return e;
      attr_set[dev] = true;
    }
  }
  const int per_window = kWindow / p.R;
  const int full = p.T / kWindow, rest = p.T % kWindow;
  const int64_t clusters = static_cast<int64_t>(full) * per_window + (rest + p.R - 1) / p.R;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * kAdCluster));
  cfg.blockDim = dim3(kAdThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kAdCluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, adapter_kernel<MT, NT>, p);
}

template <int MT>
cudaError_t launch_rank(const AdapterParams& p, cudaStream_t s) {
  if (p.r_max <= 16) return launch_shape<MT, 2>(p, s);
  if (p.r_max <= 32) return launch_shape<MT, 4>(p, s);
  return launch_shape<MT, 8>(p, s);
}

bool aligned_to(const void* p, uintptr_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

}  // namespace
}  // namespace pw

extern "C" pw_status_t pw_adapters(const uint16_t* d_x, int64_t x_stride, const uint16_t* d_a,
                                   const uint16_t* d_b, const int32_t* d_ids,
                                   const int32_t* d_ranks, const float* d_scale,
                                   int32_t n_adapters, int32_t max_rank, int32_t T, int32_t cols,
                                   int32_t rows, const void* d_base, int64_t base_stride,
                                   void* d_y, int32_t y_type, int64_t y_stride,
                                   pw_stream_t stream) {
  using namespace pw;
  auto bad = [](const char* msg) { return record_error(PW_ERR_INVALID_ARG, msg); };
  if (T < 0 || cols < 1 || rows < 1) return bad("pw_adapters: need T >= 0, cols >= 1, rows >= 1");
  if (cols > (1 << 30) || rows > (1 << 30))
    return record_error(PW_ERR_UNSUPPORTED, "pw_adapters: cols or rows above 2^30");
  if (n_adapters < 1 || n_adapters > PW_MAX_ADAPTERS)
    return bad("pw_adapters: need 1 <= n_adapters <= 4194303");
  if (max_rank < 1 || max_rank > PW_MAX_ADAPTER_RANK)
    return bad("pw_adapters: need 1 <= max_rank <= 256");
  if (y_type != PW_F32 && y_type != PW_BF16) return bad("pw_adapters: y is PW_F32 or PW_BF16");
  if (T == 0) return PW_OK;
  if (!d_x || !d_a || !d_b || !d_ids || !d_y) return bad("pw_adapters: null buffer");
  if (x_stride < 0 || base_stride < 0 || y_stride < 0 || (T > 1 && y_stride < rows))
    return bad("pw_adapters: row strides are not negative, and y's at least rows");
  if (d_base == d_y && base_stride != y_stride)
    return bad("pw_adapters: base and y in one place have one stride");
  const uintptr_t size = y_type == PW_F32 ? 4 : 2;
  if (!aligned_to(d_x, 2) || !aligned_to(d_a, 2) || !aligned_to(d_b, 2) || !aligned_to(d_ids, 4) ||
      !aligned_to(d_ranks, 4) || !aligned_to(d_scale, 4) || !aligned_to(d_base, size) ||
      !aligned_to(d_y, size))
    return bad("pw_adapters: buffers must be aligned to their elements");
  AdapterParams p{};
  p.x = d_x;
  p.a = d_a;
  p.b = d_b;
  p.ids = d_ids;
  p.ranks = d_ranks;
  p.scale = d_scale;
  p.base = d_base;
  p.y = d_y;
  p.x_ld = x_stride;
  p.base_ld = base_stride;
  p.y_ld = y_stride;
  p.n = n_adapters;
  p.r_max = max_rank;
  p.T = T;
  p.cols = cols;
  p.rows = rows;
  p.y_f32 = y_type == PW_F32;
  p.vec_x = cols % 8 == 0 && x_stride % 8 == 0 && aligned_to(d_x, 16) && aligned_to(d_a, 16);
  p.vec_b = max_rank % 4 == 0 && aligned_to(d_b, 8);
  p.vec_y = rows % 4 == 0 && y_stride % 4 == 0 && aligned_to(d_y, 4 * size) &&
            (!d_base || (base_stride % 4 == 0 && aligned_to(d_base, 4 * size)));
  // v's rows in shared memory: whole 16-rank steps; 32 or 96 bytes modulo 128
  // apart, so that the four rows of half a warp's 8-byte loads take all banks
  const int r16 = (max_rank + 15) / 16 * 16;
  p.v_ld = r16 % 32 == 0 ? r16 + 16 : r16;
  int R = 1;
  while (R < 16 && R * 37 < T) R *= 2;
  const bool wide = T >= 2048;
  p.R = wide ? 64 : R;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = wide ? launch_rank<4>(p, s) : launch_rank<1>(p, s);
  if (e != cudaSuccess) return record_error(PW_ERR_CUDA, cudaGetErrorString(e));
  return PW_OK;
}
