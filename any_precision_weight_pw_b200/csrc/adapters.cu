// adapters.cu -- pw_adapters: low-rank adapters of many requests beside one
// shared projection, y_t = base_t + scale_a * B_a (A_a x_t), a = ids[t].
//
// The tokens of a window of 256 are taken in the order of their adapters (those
// without one last), so tokens that share an adapter share its reads.
//
// Up to kNarrow tokens: one launch, a cluster of 8 blocks for each piece of at
// most 16 tokens of one adapter.  Each block takes an eighth of the columns of
// v = A x, the partial sums meet over distributed shared memory, then it takes
// an eighth of the rows of y = base + B v; B and base are in flight over the
// exchange.  Both products run on mma.sync straight from global memory: the
// contraction index may be permuted freely as long as both operands agree, so a
// lane loads 16 contiguous bytes of a row and uses them as its fragments of two
// MMA steps.  At this size the chain of dependent loads bounds the kernel, not
// the products.  (Staging through shared memory for wide tcgen05 tiles would
// lengthen the chain.)
//
// Above: two launches.  shrink_kernel leaves v of each 64 ordered tokens in the
// workspace, expand_kernel adds B v to (64 tokens) x (some 128 rows) tiles.
// Both products run on tcgen05: mma.sync did the second at a sixth of the
// tensor cores' rate and took 50 of 141 us at 4096 tokens x 14336 rows, rank 64
// (110 with tcgen05; base and y alone, 470 MB, take 93).  Measured there as a
// whole, 4096 columns, 8 requests: 117 us, 67% of the floor of 78.  The other
// bound is base and y: 512-byte runs of 64 rows, with two blocks an SM.
//
// 512 tokens are the border where both take the same time with one request a
// tile; with requests that end inside tiles the one launch wins up to 1024 (517
// tokens of 9 requests, 1409 -> 1003: 16 us against 32; 1024 of 8, 4096 ->
// 4096, rank 16: 29 against 37, rank 64: 44 against 39).
//
// Every sum has a fixed order: results do not depend on timing.
//
// Precision.  v is split into bf16 terms (v = hi + mid + lo, 24 bits; two
// terms, 16 bits, when y is bf16 and rounds to 8), each multiplied with B
// exactly; sums are fp32.  The two terms of a bf16 y save a third of the
// products and of v's shared memory; what they leave out, 2^-17 |B| |v|, shows
// only where base and B v cancel to less than 2^-8 of them.
#include <cuda_bf16.h>

#include <cmath>
#include <cstdlib>
#include <mutex>
#include <type_traits>

#include "pw_internal.h"

namespace pw {
namespace {

constexpr int kAdThreads = 256;
constexpr int kAdWarps = kAdThreads / 32;
constexpr int kAdCluster = 8;
constexpr int kWindow = 256;     // tokens ordered together
constexpr int kNarrow = 1024;    // most tokens of the one-launch path
constexpr int kTileTokens = 64;  // many tokens: tokens of a shrink cluster, of an expand tile
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
  uint8_t* ws;
  int64_t x_ld, base_ld, y_ld;
  int n, r_max, T, cols, rows;
  int per_window;  // clusters of a full window (few tokens)
  int v_ld;        // bf16 elements between the rows of v
  int n_terms;     // bf16 terms of v
  int r32;         // max_rank in whole 32s
  int tile_rows;   // many tokens: rows of an expand tile
  int split;       // and blocks of a shrink cluster
  unsigned long long wait_ns;  // limit of a wait
  int stall_tile;  // test switch: this tile's products are not issued (-1: none;
                   // in expand -2 - tile)
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

// 8 bf16 from column c of a row of `cols`, zero past the row; VEC: the row and
// c are 16-byte aligned, cols % 8 == 0
template <bool VEC>
__device__ __forceinline__ uint4 load8(const uint16_t* row, int c, int cols) {
  const uint16_t* p = row + c;
  const int count = cols - c;
  if (count <= 0) return make_uint4(0, 0, 0, 0);
  if constexpr (VEC) return __ldg(reinterpret_cast<const uint4*>(p));
  if (c >= 3 && count >= 12) {
    // inside the row at any alignment: the three aligned 8-byte words around
    // the 16 bytes, shifted by whole and half words
    const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 7;
    const uint2* w = reinterpret_cast<const uint2*>(reinterpret_cast<uintptr_t>(p) - off);
    const uint2 w0 = __ldg(w), w1 = __ldg(w + 1), w2 = __ldg(w + 2);
    const bool one = off & 4;
    const uint32_t a = one ? w0.y : w0.x, b = one ? w1.x : w0.y, d = one ? w1.y : w1.x,
                   e = one ? w2.x : w1.y, f = one ? w2.y : w2.x;
    const uint32_t s = (off & 2) * 8;
    return make_uint4(__funnelshift_r(a, b, s), __funnelshift_r(b, d, s), __funnelshift_r(d, e, s),
                      __funnelshift_r(e, f, s));
  }
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = i < count ? __ldg(p + i) : 0u;
  return make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
}
// 8 bf16 from rank k of a row of B, zero from `rank` on; VEC: k is 16-byte
// aligned in a row of whole 16-byte pieces
template <bool VEC>
__device__ __forceinline__ uint4 load_ranks(const uint16_t* row, int k, int rank) {
  if constexpr (!VEC) return load8<false>(row, k, rank);
  const int count = rank - k;
  uint4 v = make_uint4(0, 0, 0, 0);
  if (count > 0) v = __ldg(reinterpret_cast<const uint4*>(row + k));
  if (rank & 7) {  // the same for the warp
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] &= count >= 2 * i + 2 ? 0xffffffffu : count == 2 * i + 1 ? 0xffffu : 0u;
    v = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return v;
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

// Window order in shared memory: position -> token of the window and adapter
// (-1 for none, behind the others).  All 256 threads; key: scratch.  Windows
// whose runs are long as they are stay so if keep_runs.
__device__ __forceinline__ void order_window(const AdapterParams& p, int t0, int n_win,
                                             bool keep_runs, int* key, int* tok, int* sid) {
  const int tid = threadIdx.x;
  int id = -1;
  if (tid < n_win) {
    id = p.ids[t0 + tid];
    if (id < 0 || id >= p.n) id = -1;
  }
  // no adapter: 2^22 - 1, above every other; the position in the low 8 bits
  const int k = ((id < 0 ? PW_MAX_ADAPTERS : id) << 8) | tid;
  key[tid] = tid < n_win ? k : INT32_MAX;
  __syncthreads();
  const bool change = tid > 0 && tid < n_win && (key[tid - 1] >> 8) != (k >> 8);
  const int runs = 1 + __syncthreads_count(change);
  int pos = tid;
  if (keep_runs ? runs * 16 > n_win : runs > 1) {  // position = number of smaller keys
    pos = 0;
    for (int i = 0; i < n_win; i += 4) {
      const int4 k4 = *reinterpret_cast<const int4*>(key + i);
      pos += (k4.x < k) + (k4.y < k) + (k4.z < k) + (k4.w < k);
    }
  }
  if (tid < n_win) {
    tok[pos] = t0 + tid;
    sid[pos] = id;
  }
  __syncthreads();
}

__device__ __forceinline__ int adapter_rank(const AdapterParams& p, int id) {
  if (id < 0) return 0;
  return p.ranks ? min(max(p.ranks[id], 0), p.r_max) : p.r_max;
}

// ---- the two products --------------------------------------------------------

// Partial sums of a piece's v for ranks [r0, r0 + 8 NT) over the 32-column
// blocks kb0, kb0 + step, ... < kb1.  tok: the piece's tokens.
template <bool VEC, int NT>
__device__ __forceinline__ void shrink_acc(const AdapterParams& p, const Piece& pc, const int* tok,
                                           int r0, int kb0, int kb1, int step, float (&acc)[NT][4]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int nr = pc.rank - r0;
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
  if (nr <= 0) return;
  const int c0 = g < pc.len ? p.cols : 0, c1 = g + 8 < pc.len ? p.cols : 0;  // columns there are
  const uint16_t* x0 = p.x + (c0 ? tok[g] : 0) * p.x_ld;
  const uint16_t* x1 = p.x + (c1 ? tok[g + 8] : 0) * p.x_ld;
  const uint16_t* ar = p.a + (static_cast<int64_t>(pc.adapter) * p.r_max + r0 + g) * p.cols;
#pragma unroll (NT == 8 ? 1 : 2)
  for (int kb = kb0; kb < kb1; kb += step) {
    const int c = kb * 32 + q * 8;
    const uint4 xa = load8<VEC>(x0, c, c0);
    const uint4 xb = load8<VEC>(x1, c, c1);
    uint4 w[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j)
      w[j] = load8<VEC>(ar + static_cast<int64_t>(8 * j) * p.cols, c, 8 * j + g < nr ? p.cols : 0);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      mma16816(acc[j], xa.x, xb.x, xa.y, xb.y, w[j].x, w[j].y);
      mma16816(acc[j], xa.z, xb.z, xa.w, xb.w, w[j].z, w[j].w);
    }
  }
}

// acc of a warp to its [16][8 NT] tile in shared memory
template <int NT>
__device__ __forceinline__ void store_acc(float* tile, const float (&acc)[NT][4]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    *reinterpret_cast<float2*>(tile + g * 8 * NT + 8 * j + 2 * q) = make_float2(acc[j][0], acc[j][1]);
    *reinterpret_cast<float2*>(tile + (g + 8) * 8 * NT + 8 * j + 2 * q) =
        make_float2(acc[j][2], acc[j][3]);
  }
}

// The next bf16 term of two neighbouring values, as one word.  Infinities and
// NaN are whole in the first.
__device__ __forceinline__ uint32_t next_term(float (&v)[2]) {
  uint16_t h[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    h[i] = bf16_bits(v[i]);
    const float hv = bf16_value(h[i]);
    v[i] = fabsf(hv) < INFINITY ? v[i] - hv : 0.f;
  }
  return h[0] | static_cast<uint32_t>(h[1]) << 16;
}

// 16 tokens x 16 rows of the second product, y = base - B (-v): v is kept
// negated, so that a sum of nothing, +0, leaves base as it is, -0 too.  MMA
// column g of tile j is row o + 4 (g / 2) + 2 j + g % 2: a lane then holds rows
// 4q..4q+3, whole 16-byte accesses of base and y.  A lane holds ranks 8q..8q+7
// of each 32 (two MMA steps), whole 16-byte accesses of B and v.
// KS: 32-rank steps.  F32: type of base and y.  VEC: every access is aligned.
template <int KS, bool F32, bool VEC>
struct ExpandTile {
  static constexpr int kTerms = F32 ? 3 : 2;
  using E = typename std::conditional<F32, float, uint16_t>::type;
  using Raw4 = typename std::conditional<F32, float4, uint2>::type;

  // A lane's tokens (rows g and g + 8 of the piece) and its place in B and v.
  struct Lane {
    const E* base[2];
    E* y[2];
    const uint16_t* b;  // row 4 (g / 2) + g % 2 of the adapter
    const uint16_t* v;
    bool on[2], any_base;
    int left;           // rows from this lane's first on
    __device__ __forceinline__ Lane(const AdapterParams& p, const Piece& pc, const int* tok,
                                    const uint16_t* v_rows) {
      const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        on[h] = g + 8 * h < pc.len;
        const int64_t t = on[h] ? tok[g + 8 * h] : 0;
        base[h] = static_cast<const E*>(p.base) + t * p.base_ld + 4 * q;
        y[h] = static_cast<E*>(p.y) + t * p.y_ld + 4 * q;
      }
      any_base = p.base != nullptr;
      b = p.b + (static_cast<int64_t>(max(pc.adapter, 0)) * p.rows + 4 * (g >> 1) + (g & 1)) * p.r_max;
      v = v_rows + g * p.v_ld + 8 * q;
      left = p.rows - 4 * q;
    }
  };

  Raw4 add[2];     // [token half]: base as it lies in memory
  uint4 w[KS][2];  // B

  // base, and B of ranks [0, 32 KS)
  __device__ __forceinline__ void load(const AdapterParams& p, const Piece& pc, const Lane& l, int ob) {
    const int left = l.left - ob * 16;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const E* src = l.base[h] + ob * 16;
      Raw4 r = {};
      if (l.any_base && l.on[h] && left > 0) {
        if constexpr (VEC) {
          r = *reinterpret_cast<const Raw4*>(src);
        } else {
          E e[4] = {src[0], left > 1 ? src[1] : E(0), left > 2 ? src[2] : E(0),
                    left > 3 ? src[3] : E(0)};
          if constexpr (F32)
            r = make_float4(e[0], e[1], e[2], e[3]);
          else
            r = make_uint2(e[0] | static_cast<uint32_t>(e[1]) << 16,
                           e[2] | static_cast<uint32_t>(e[3]) << 16);
        }
      }
      add[h] = r;
    }
    load_b(p, pc, l, ob, 0);
  }
  __device__ __forceinline__ void load_b(const AdapterParams& p, const Piece& pc, const Lane& l,
                                         int ob, int k0) {
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int rows = p.rows - ob * 16 - 4 * (g >> 1) - (g & 1);
    const uint16_t* src = l.b + static_cast<int64_t>(ob * 16) * p.r_max;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
        w[ks][j] = load_ranks<VEC>(src + 2 * j * p.r_max, k0 + 32 * ks + 8 * q,
                                   rows > 2 * j ? pc.rank : 0);
  }
  // left: ranks from k0 on
  __device__ __forceinline__ void multiply(const AdapterParams& p, const Lane& l, int v_plane, int k0,
                                           int left, float (&acc)[2][4]) const {
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      if (32 * ks >= left) break;
#pragma unroll
      for (int t = 0; t < kTerms; ++t) {
        const uint16_t* vp = l.v + t * v_plane + k0 + 32 * ks;
        const uint4 lo = *reinterpret_cast<const uint4*>(vp);
        const uint4 hi = *reinterpret_cast<const uint4*>(vp + 8 * p.v_ld);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          mma16816(acc[j], lo.x, hi.x, lo.y, hi.y, w[ks][j].x, w[ks][j].y);
          mma16816(acc[j], lo.z, hi.z, lo.w, hi.w, w[ks][j].z, w[ks][j].w);
        }
      }
    }
  }
  __device__ __forceinline__ void store(const Lane& l, int ob, const float (&acc)[2][4]) const {
    const int left = l.left - ob * 16;
    if (left <= 0) return;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (!l.on[h]) continue;
      const Raw4 r = add[h];
      float v[4];
      if constexpr (F32) {
        v[0] = r.x, v[1] = r.y, v[2] = r.z, v[3] = r.w;
      } else {
        v[0] = __uint_as_float(r.x << 16), v[1] = __uint_as_float(r.x & 0xffff0000u);
        v[2] = __uint_as_float(r.y << 16), v[3] = __uint_as_float(r.y & 0xffff0000u);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] -= acc[i >> 1][2 * h + (i & 1)];
      E* dst = l.y[h] + ob * 16;
      if constexpr (VEC) {
        if constexpr (F32)
          *reinterpret_cast<float4*>(dst) = make_float4(v[0], v[1], v[2], v[3]);
        else
          *reinterpret_cast<uint2*>(dst) =
              make_uint2(bf16_bits(v[0]) | static_cast<uint32_t>(bf16_bits(v[1])) << 16,
                         bf16_bits(v[2]) | static_cast<uint32_t>(bf16_bits(v[3])) << 16);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < left) {
            if constexpr (F32)
              dst[i] = v[i];
            else
              dst[i] = bf16_bits(v[i]);
          }
      }
    }
  }
};

// The second product of one piece over 16-row blocks ob, ob + step, ... < ob1,
// D tiles in flight.  Ranks above 32 KS take further steps (MULTI).
template <int D, bool MULTI, int KS, bool F32, bool VEC>
struct Expand {
  using Tile = ExpandTile<KS, F32, VEC>;
  Tile t[D];
  __device__ __forceinline__ void start(const AdapterParams& p, const Piece& pc,
                                        const typename Tile::Lane& l, int ob, int ob1, int step) {
#pragma unroll
    for (int d = 0; d < D; ++d)
      if (ob + d * step < ob1) t[d].load(p, pc, l, ob + d * step);
  }
  __device__ __forceinline__ void run(const AdapterParams& p, const Piece& pc,
                                      const typename Tile::Lane& l, int v_plane, int ob, int ob1,
                                      int step) {
    while (ob < ob1) {
#pragma unroll
      for (int d = 0; d < D; ++d, ob += step) {
        if (ob >= ob1) return;
        float acc[2][4] = {};
        t[d].multiply(p, l, v_plane, 0, pc.rank, acc);
        if (MULTI)
          for (int k0 = 32 * KS; k0 < pc.rank; k0 += 32 * KS) {
            t[d].load_b(p, pc, l, ob, k0);
            t[d].multiply(p, l, v_plane, k0, pc.rank - k0, acc);
          }
        t[d].store(l, ob, acc);
        if (ob + D * step < ob1) t[d].load(p, pc, l, ob + D * step);
      }
    }
  }
};

// ---- few tokens: one launch, a cluster per piece -----------------------------

template <int NT, bool MULTI, bool F32, bool VEC>
__global__ void __launch_bounds__(kAdThreads, 2) adapter_kernel(const AdapterParams p) {
  constexpr int kChunk = 8 * NT;       // ranks of a shrink step
  constexpr int kTile = 16 * kChunk;   // sums of a piece and step
  constexpr int KS = NT == 8 ? 2 : 1;
  extern __shared__ __align__(16) uint8_t smem[];
  float* red = reinterpret_cast<float*>(smem);  // [8 warps][16][kChunk]
  float* slots = red + kAdWarps * kTile;        // [1, MULTI 2][8 blocks][16][kChunk]
  uint16_t* vt = reinterpret_cast<uint16_t*>(slots + (MULTI ? 2 : 1) * kAdCluster * kTile);
  __shared__ __align__(16) int s_key[kWindow];
  __shared__ int s_tok[kWindow], s_sid[kWindow];
  __shared__ uint32_t s_mask[2][kAdWarps];
  __shared__ Piece s_piece;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(cluster_rank());
  const int cl = blockIdx.x / kAdCluster;
  const int t0 = cl / p.per_window * kWindow;  // the window's first token
  const int n_win = min(kWindow, p.T - t0);
  const int want = cl % p.per_window;          // this cluster's piece
  pdl_wait();

  if (p.T == 1) {
    if (tid == 0) {
      const int id = p.ids[0], a = id >= 0 && id < p.n ? id : -1;
      s_tok[0] = 0;
      s_piece = {0, 1, a, adapter_rank(p, a)};
    }
    __syncthreads();
  } else {
    order_window(p, t0, n_win, false, s_key, s_tok, s_sid);
    if (tid == 0) s_piece = {0, 0, -1, 0};
    // a piece starts where the adapter changes and at every 16th token of a run
    const bool change = tid < n_win && (tid == 0 || s_sid[tid] != s_sid[tid - 1]);
    const uint32_t cm = __ballot_sync(0xffffffffu, change);
    if (lane == 0) s_mask[0][warp] = cm;
    __syncthreads();
    int run = 0;
    for (int w = warp; w >= 0; --w) {
      const uint32_t m = s_mask[0][w] & (w == warp ? 0xffffffffu >> (31 - lane) : 0xffffffffu);
      if (m) {
        run = w * 32 + 31 - __clz(m);
        break;
      }
    }
    const bool start = tid < n_win && (tid - run) % 16 == 0;
    const uint32_t sm = __ballot_sync(0xffffffffu, start);
    if (lane == 0) s_mask[1][warp] = sm;
    __syncthreads();
    if (start) {
      int index = __popc(sm & ((1u << lane) - 1));
      for (int w = 0; w < warp; ++w) index += __popc(s_mask[1][w]);
      if (index == want) {
        int end = n_win;
        for (int w = warp; w < kAdWarps; ++w) {
          const uint32_t m = s_mask[1][w] & (w > warp    ? 0xffffffffu
                                             : lane == 31 ? 0u
                                                          : 0xffffffffu << (lane + 1));
          if (m) {
            end = w * 32 + __ffs(m) - 1;
            break;
          }
        }
        s_piece = {tid, end - tid, s_sid[tid], adapter_rank(p, s_sid[tid])};
      }
    }
    __syncthreads();
  }
  const Piece pc = s_piece;  // the same in all blocks of the cluster
  if (pc.len == 0 || (pc.rank == 0 && p.base == p.y)) return;
  const int* tok = s_tok + pc.start;
  if (pc.rank > 0) cluster_arrive();  // the others' shared memory is live once all have arrived

  // this block's columns (shrink, in 32s) and rows (expand, in 16s)
  const int kb_all = (p.cols + 31) / 32, ob_all = (p.rows + 15) / 16;
  const int kb0 = rank * kb_all / kAdCluster, kb1 = (rank + 1) * kb_all / kAdCluster;
  const int ob0 = rank * ob_all / kAdCluster + warp, ob1 = (rank + 1) * ob_all / kAdCluster;
  const int v_plane = 16 * p.v_ld;
  const float minus = pc.adapter >= 0 && p.scale ? -p.scale[pc.adapter] : -1.f;

  using Tile = ExpandTile<KS, F32, VEC>;
  const typename Tile::Lane l(p, pc, tok, vt);
  Expand<MULTI ? 1 : KS == 2 ? 3 : 4, MULTI, KS, F32, VEC> second;
  if (pc.rank == 0) second.start(p, pc, l, ob0, ob1, kAdWarps);
  auto shrink = [&](int r0, int step) {
    float acc[NT][4];
    shrink_acc<VEC, NT>(p, pc, tok, r0, kb0 + warp, kb1, kAdWarps, acc);
    store_acc<NT>(red + warp * kTile, acc);
    if (r0 == 0) {
      second.start(p, pc, l, ob0, ob1, kAdWarps);  // in flight over the exchange
      cluster_wait();
    }
    __syncthreads();
    // this block's sums to every block, rows in use only
    float* slot = slots + (MULTI ? (step & 1) * kAdCluster * kTile : 0);
    for (int e = tid * 4; e < pc.len * kChunk; e += kAdThreads * 4) {
      float4 s = *reinterpret_cast<const float4*>(red + e);
#pragma unroll
      for (int k = 1; k < kAdWarps; ++k) {
        const float4 o = *reinterpret_cast<const float4*>(red + k * kTile + e);
        s.x += o.x, s.y += o.y, s.z += o.z, s.w += o.w;
      }
      const uint32_t d = smem_u32(slot + rank * kTile + e);
#pragma unroll
      for (int c = 0; c < kAdCluster; ++c) put4(in_block(d, c), s);
    }
    cluster_arrive();
    cluster_wait();
    // sums over the blocks; scale v, negate it and split it into bf16 terms
    for (int e = tid * 2; e < pc.len * kChunk; e += kAdThreads * 2) {
      const int row = e / kChunk, k = r0 + e % kChunk;
      if (k >= p.r32) continue;
      float v[2] = {0.f, 0.f};
#pragma unroll
      for (int c = 0; c < kAdCluster; ++c) {
        const float2 o = *reinterpret_cast<const float2*>(slot + c * kTile + e);
        v[0] += o.x, v[1] += o.y;
      }
      // from the adapter's rank on v is zero, also where x or the scale is not
      // finite (inf times the zeros read for A there is NaN)
      v[0] = k < pc.rank ? v[0] * minus : 0.f;
      v[1] = k + 1 < pc.rank ? v[1] * minus : 0.f;
#pragma unroll
      for (int t = 0; t < Tile::kTerms; ++t) {
        uint16_t* d = vt + t * v_plane + row * p.v_ld + k;
        *reinterpret_cast<uint32_t*>(d) = next_term(v);
        if (kChunk == 16) *reinterpret_cast<uint32_t*>(d + 16) = 0;
      }
    }
    __syncthreads();
  };
  if (pc.rank > 0) {
    shrink(0, 0);
    if constexpr (MULTI)
      for (int r0 = kChunk, step = 1; r0 < pc.rank; r0 += kChunk, ++step) shrink(r0, step);
  }
  second.run(p, pc, l, v_plane, ob0, ob1, kAdWarps);
}

// ---- many tokens: shrink, then expand ----------------------------------------

// What shrink leaves for expand, per 64 tokens: the segments (neighbours of
// one adapter), the tokens, and v (n_terms planes of [64][v_ld] bf16, by
// position, zero from the rank on to the next multiple of 32).
struct alignas(16) TileInfo {  // moved in 16-byte pieces, in shared memory too
  int n_segments, pad[3];
  Piece segment[kTileTokens];
  int tok[kTileTokens];
};
static_assert(alignof(TileInfo) == alignof(uint4) && sizeof(TileInfo) % sizeof(uint4) == 0,
              "TileInfo is copied as uint4");
static_assert(sizeof(TileInfo) / sizeof(uint4) <= kAdThreads, "one piece a thread");
__host__ __device__ __forceinline__ int64_t tile_bytes(int n_terms, int v_ld) {
  return static_cast<int64_t>(sizeof(TileInfo)) + 2ll * n_terms * kTileTokens * v_ld;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t pred = 0;
  asm volatile(
      "{\n.reg .pred P1;\n.reg .b32 r;\nelect.sync r|P1, %1;\nselp.u32 %0, 1, 0, P1;\n}\n"
      : "=r"(pred)
      : "r"(0xffffffffu));
  return pred != 0;
}
// K-major operand in 128-byte swizzle: 64 bf16 a row, 8-row groups of 1024
// bytes, 16-byte piece c of row r at piece c ^ (r & 7).
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | 1ull << 16 | 64ull << 32 | 1ull << 46 |
         2ull << 61;
}
__device__ __forceinline__ uint32_t operand_off(int row, int piece) {
  return (row >> 3) * 1024 + (row & 7) * 128 + ((piece ^ (row & 7)) << 4);
}
// bf16 x bf16 -> fp32, M = 128
__device__ __forceinline__ uint32_t mma_idesc(int n) {
  return 1u << 4 | 1u << 7 | 1u << 10 | static_cast<uint32_t>(n >> 3) << 17 | 8u << 24;
}
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t acc) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc));
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
  uint32_t* u = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, "
      "%29, %30, %31}, [%32];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]),
        "=r"(u[7]), "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]),
        "=r"(u[14]), "=r"(u[15]), "=r"(u[16]), "=r"(u[17]), "=r"(u[18]), "=r"(u[19]),
        "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]), "=r"(u[25]),
        "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
// Wait for an mbarrier phase, limit_ns at most; a wait that gives up makes the
// block's later ones give up at once.
__device__ __forceinline__ void mbar_wait(uint32_t bar, uint32_t parity, volatile int* gave_up,
                                          unsigned long long limit_ns) {
  unsigned long long t0 = 0, t = 0;
  while (true) {
    uint32_t ok;
    asm volatile(
        "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        "selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok || *gave_up) return;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    if (t0 == 0) t0 = t;
    if (t - t0 > limit_ns) {
      *gave_up = 1;
      return;
    }
  }
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t* u = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15}, [%16];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]),
        "=r"(u[7]), "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]),
        "=r"(u[14]), "=r"(u[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// What is written where a wait gave up.
__device__ __forceinline__ float lost_value() { return __int_as_float(0x7fffffff); }

// Before tensor memory goes back after a wait that gave up: the products still
// in flight, waited for once more (all threads).
__device__ __forceinline__ void drain_products(uint32_t bar, unsigned long long limit_ns) {
  if (threadIdx.x >= 32) return;
  if (elect_one())
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
        : "memory");
  __syncwarp();
  int again = 0;
  mbar_wait(bar, 0, &again, limit_ns);
}

constexpr int kShrinkStages = 3;
constexpr int kShrinkStage = 3 * 64 * 128;  // bytes: x [64][64], A [64][64] of two segments
constexpr int kChains = 4;                  // accumulators the steps of a pass go to in turn
constexpr int kTmemCols = 64 * kChains;

// v of 64 ordered tokens: a cluster of p.split blocks, each its share of the
// columns.  A pass takes two neighbouring segments and 64 ranks: D[token][rank]
// = x [64][64] A_s^T over the block's 64-column steps on tcgen05, x once for
// both, copied two steps ahead; a token takes its own segment's D (tiles on the
// border of two requests in one pass: the operator 133 -> 117 us at 4096 tokens
// of 8 requests, 4096 -> 14336, rank 64).  The MMA has 128 rows; the upper 64 run over the A tile behind x
// and are not used (the tensor cores have the time).  Partial sums go to the
// block that owns the tokens, which adds them in rank order.  The tensor cores
// cut their sums off instead of rounding them: the steps go to two (two
// segments) or four accumulators in turn, which keeps the chains short (one:
// 1.1e-6 relative error of y at 4096 columns and rank 64).
template <bool VEC>
__global__ void __launch_bounds__(kAdThreads, 2) shrink_kernel(const AdapterParams p) {
  constexpr int STAGES = kShrinkStages;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ __align__(16) float slots[kTileTokens * 64];  // [block][own token][rank]
  __shared__ __align__(16) int s_key[kWindow];
  __shared__ int s_tok[kWindow], s_sid[kWindow];
  __shared__ TileInfo s_info;
  __shared__ __align__(8) uint64_t s_bar[3];  // products of even and odd steps; the end, after a lost wait
  __shared__ uint32_t s_tmem;
  __shared__ int s_gave_up;
  const uint32_t sm = (smem_u32(smem) + 1023) & ~1023u;
  uint8_t* const smp = smem + (sm - smem_u32(smem));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(cluster_rank());
  const int split = p.split, own = kTileTokens / split;  // blocks; tokens a block owns
  const int cl = blockIdx.x / split;
  constexpr int kPerWindow = kWindow / kTileTokens;
  const int t0 = cl / kPerWindow * kWindow;
  const int n_win = min(kWindow, p.T - t0);
  const int first = cl % kPerWindow * kTileTokens;
  const int n_rows = min(kTileTokens, n_win - first);  // >= 1 by the grid
  const uint32_t bar = smem_u32(s_bar);
  cluster_arrive();  // the others' shared memory is live once all have arrived
  pdl_wait();
  pdl_trigger();  // expand's blocks may start; they wait for this grid's end
  if (tid == 0) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(bar));
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(bar + 8));
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(bar + 16));
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    s_gave_up = 0;
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&s_tmem)),
                 "r"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  order_window(p, t0, n_win, true, s_key, s_tok, s_sid);
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const int* tok = s_tok + first;
  const int* sid = s_sid + first;
  if (warp == 0) {
    uint64_t changes = 0;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int i = lane + 32 * half;
      const bool c = i < n_rows && (i == 0 || sid[i] != sid[i - 1]);
      changes |= static_cast<uint64_t>(__ballot_sync(0xffffffffu, c)) << (32 * half);
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int i = lane + 32 * half;
      if (i < n_rows) s_info.tok[i] = tok[i];
      if (!(changes >> i & 1)) continue;
      const uint64_t above = i == 63 ? 0ull : changes & (~0ull << (i + 1));
      s_info.segment[__popcll(changes & ((1ull << i) - 1))] = {
          i, (above ? __ffsll(above) - 1 : n_rows) - i, sid[i], adapter_rank(p, sid[i])};
    }
    if (lane == 0) s_info.n_segments = __popcll(changes);
  }
  __syncthreads();
  uint8_t* ws = p.ws + cl * tile_bytes(p.n_terms, p.v_ld);
  if (rank == 0 && tid < static_cast<int>(sizeof(TileInfo) / 16))
    reinterpret_cast<uint4*>(ws)[tid] = reinterpret_cast<const uint4*>(&s_info)[tid];
  uint16_t* vt = reinterpret_cast<uint16_t*>(ws + sizeof(TileInfo));
  const int v_plane = kTileTokens * p.v_ld;
  const int kb_all = (p.cols + 63) / 64;
  const int kb0 = static_cast<int>(static_cast<int64_t>(rank) * kb_all / split);
  const int kb1 = static_cast<int>(static_cast<int64_t>(rank + 1) * kb_all / split);
  const int n_segments = s_info.n_segments, n_steps = kb1 - kb0;
  // A pass: segments g0 and g0 + 1 of the tile, ranks [r0, r0 + 64).
  struct Pass {
    int start, len, len0;  // tokens of both, of the first
    int rank[2], adapter[2];
  };
  auto pass_of = [&](int g0) {
    const Piece s0 = s_info.segment[g0];
    Pass w = {s0.start, s0.len, s0.len, {s0.rank, 0}, {s0.adapter, -1}};
    if (g0 + 1 < n_segments) {
      const Piece s1 = s_info.segment[g0 + 1];
      w.len += s1.len;
      w.rank[1] = s1.rank;
      w.adapter[1] = s1.adapter;
    }
    return w;
  };
  // The copies run ahead over the passes, with their own place: rows `row` and
  // row + 32 of the three tiles, one 16-byte piece of each step.
  const int row = tid >> 3, pc = tid & 7;
  const uint32_t off = operand_off(row, pc);  // row + 32: 4096 behind; the next tile: 8192
  int l_g0 = 0, l_r0 = 0, l_i = 0, l_stage = 0, l_col = 0, l_rank = 0;
  const uint16_t* l_src[6] = {};  // x, A of the first, of the second; row and row + 32
  bool l_on[6] = {};
  auto issue = [&]() {
    while (l_i == 0 && l_r0 == 0 && l_g0 < n_segments) {  // the next pair with a rank
      const Pass w = pass_of(l_g0);
      l_rank = max(w.rank[0], w.rank[1]);
      if (l_rank > 0) break;
      l_g0 += 2;
    }
    if (l_g0 < n_segments) {
      if (l_i == 0) {
        const Pass w = pass_of(l_g0);
        l_col = kb0 * 64 + pc * 8;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = row + 32 * h;
          l_on[h] = r < w.len;
          l_src[h] = p.x + tok[w.start + min(r, w.len - 1)] * p.x_ld;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            l_on[2 + 2 * j + h] = l_r0 + r < w.rank[j];
            l_src[2 + 2 * j + h] =
                p.a + (static_cast<int64_t>(max(w.adapter[j], 0)) * p.r_max + l_r0 + r) * p.cols;
          }
        }
      }
      const uint32_t at = l_stage * kShrinkStage + off;
#pragma unroll
      for (int h = 0; h < 6; ++h)
        if (l_on[h]) {
          if constexpr (VEC)
            cp_async16(sm + at + h * 4096, l_col < p.cols ? l_src[h] + l_col : p.x,
                       l_col < p.cols ? 16 : 0);
          else
            *reinterpret_cast<uint4*>(smp + at + h * 4096) = load8<false>(l_src[h], l_col, p.cols);
        }
      l_col += 64;
      l_stage = l_stage + 1 == STAGES ? 0 : l_stage + 1;
      if (++l_i == n_steps) {
        l_i = 0;
        l_r0 += 64;
        if (l_r0 >= l_rank) {
          l_r0 = 0;
          l_g0 += 2;
        }
      }
    }
    __syncwarp();
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (n_steps > 0)
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) issue();
  cluster_wait();
  // Steps so far.  A step's wait comes after the next one's products have been
  // issued, hence two barriers: one would be two phases ahead of it.
  uint32_t n_done = 0;
  auto wait_step = [&](uint32_t n) { mbar_wait(bar + (n & 1) * 8, n >> 1 & 1, &s_gave_up, p.wait_ns); };
  int stage = 0;
  bool sums_read = false;  // an arrive without its wait: this block has read its sums
  for (int g0 = 0; g0 < n_segments; g0 += 2) {
    const Pass w = pass_of(g0);
    float sc[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
      sc[j] = w.adapter[j] >= 0 && p.scale ? p.scale[w.adapter[j]] : 1.f;
    for (int r0 = 0; r0 < max(w.rank[0], w.rank[1]); r0 += 64) {
      const int n_r[2] = {min(64, w.rank[0] - r0), min(64, w.rank[1] - r0)};  // none if <= 0
      // accumulators: chain c of segment j at 64 (per * j + c)
      const int per = n_r[0] > 0 && n_r[1] > 0 ? kChains / 2 : kChains;
      const int second = per == kChains ? 0 : 64 * per;
      for (int i = 0; i < n_steps; ++i) {
        asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncthreads();  // the step is there
        if (warp == 0 && cl != p.stall_tile) {
          tc_fence_after();
          if (elect_one()) {
            const uint32_t at = sm + stage * kShrinkStage;
            const uint64_t dx = operand_desc(at);
            const uint32_t d = tmem + i % per * 64;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              if (n_r[j] <= 0) continue;
              const uint64_t da = operand_desc(at + 8192 * (1 + j));
              const uint32_t idesc = mma_idesc((n_r[j] + 15) / 16 * 16);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                tc_mma(d + j * second, dx + 2 * k, da + 2 * k, idesc, i >= per || k > 0);
            }
            asm volatile(
                "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                    bar + (n_done & 1) * 8)
                : "memory");
          }
          __syncwarp();
        }
        stage = stage + 1 == STAGES ? 0 : stage + 1;
        if (i > 0) wait_step(n_done - 1);  // its stage takes the next copies
        ++n_done;
        issue();
      }
      if (n_steps > 0) wait_step(n_done - 1);
      if (sums_read) cluster_wait();  // the last sums have been read everywhere
      // token 32 warp + lane of its segment's accumulators to its owner
      if (warp < 2 && warp * 32 < w.len) {
        const int t = warp * 32 + lane;
        const uint32_t d = in_block(smem_u32(slots + (rank * own + t % own) * 64), t / own);
        tc_fence_after();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float v[32] = {};
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            // the same for the warp: the segment has ranks here and tokens among these 32
            if (32 * h >= n_r[j] || (j == 0 ? warp * 32 >= w.len0 : warp * 32 + 32 <= w.len0)) continue;
            const bool mine = (t >= w.len0) == (j == 1);
            for (int c = 0; c < min(n_steps, per); ++c) {
              float u[32];
              tmem_ld32(tmem + (static_cast<uint32_t>(warp) * 32 << 16) + j * second + c * 64 + 32 * h, u);
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] = mine ? v[e] + u[e] : v[e];
            }
          }
          if (*static_cast<volatile int*>(&s_gave_up)) {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = lost_value();
          }
          if (t < w.len)
#pragma unroll
            for (int e = 0; e < 8; ++e)
              put4(d + (32 * h + 4 * e) * 4,
                   make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]));
        }
        tc_fence_before();
      }
      cluster_arrive();
      cluster_wait();
      // sums over the blocks; scale v and split it into bf16 terms
      for (int e = tid * 2; e < own * 64; e += kAdThreads * 2) {
        const int t = rank * own + e / 64, k = e % 64;
        const bool two = t >= w.len0;
        const int n = two ? n_r[1] : n_r[0];
        if (t >= w.len || n <= 0 || r0 + k >= p.r32) continue;
        float v[2] = {0.f, 0.f};
        for (int c = 0; c < split; ++c) {
          const float2 u = *reinterpret_cast<const float2*>(slots + c * own * 64 + e);
          v[0] += u.x, v[1] += u.y;
        }
        const float f = two ? sc[1] : sc[0];
        v[0] = k < n ? v[0] * f : 0.f;
        v[1] = k + 1 < n ? v[1] * f : 0.f;
        for (int i = 0; i < p.n_terms; ++i)
          *reinterpret_cast<uint32_t*>(vt + i * v_plane + (w.start + t) * p.v_ld + r0 + k) =
              next_term(v);
      }
      // relaxed: nothing is handed over (a release would wait for v's stores)
      asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
      sums_read = true;
    }
  }
  if (sums_read) cluster_wait();
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  if (s_gave_up) drain_products(bar + 16, p.wait_ns);
  tc_fence_after();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
}

constexpr int kBlk = 128;          // rows (of W) of an expand step
constexpr int kVTile = 64 * 128;   // bytes of 64 ranks of v
constexpr int kBTile = 128 * 128;  // of B
constexpr int kExpandStages = 3;

// y = base + B v over (64 tokens) x (tile_rows rows) tiles, 128 rows at a time:
// D_s[row][token] = B_s [128][rank] x v^T [rank][64] on tcgen05 for each of up
// to kGroup neighbouring segments s of the tile, one product per bf16 term of v
// into the segment's accumulator; a token takes its own segment's column.  (A
// tile on the border of two requests then reads and writes its tokens once, and
// values of one adapter never meet another's tokens.)  The product is taken
// this way round because tensor memory hands each lane one row of D: a warp's
// 32 lanes then hold 32 neighbouring rows of W for a token, and base and y move
// in runs of 128 bytes (fp32; bf16 64) at any alignment.  B is copied to shared memory
// asynchronously in steps of 64 ranks, STAGES - 1 steps ahead; base is loaded
// 128 rows ahead into registers.
// NC: 64-rank steps at most.  VEC: 16-byte copies of B are legal.
constexpr int kGroup = 4;
constexpr int kExpandCols = 64 * kGroup;
template <int NC, bool F32, bool VEC>
__global__ void __launch_bounds__(kAdThreads, NC == 1 ? 2 : 1) expand_kernel(const AdapterParams p) {
  constexpr int STAGES = kExpandStages, kTerms = F32 ? 3 : 2;
  using E = typename std::conditional<F32, float, uint16_t>::type;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ TileInfo s_info;
  __shared__ int64_t s_base[kTileTokens], s_y[kTileTokens];  // byte offsets of the segment's tokens
  __shared__ __align__(8) uint64_t s_bar[2];  // products; the end, after a lost wait
  __shared__ uint32_t s_tmem;
  __shared__ int s_gave_up;
  const uint32_t sm = (smem_u32(smem) + 1023) & ~1023u;  // v: [term][step], then the stages of B
  uint8_t* const smp = smem + (sm - smem_u32(smem));
  const uint32_t st0 = kTerms * NC * kVTile;             // offset of the stages
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n_chunks = (p.rows + p.tile_rows - 1) / p.tile_rows;
  const int64_t tile = blockIdx.x / n_chunks;
  const int first = blockIdx.x % n_chunks * p.tile_rows;  // the block's rows
  const int rows = min(p.rows - first, p.tile_rows), nb = (rows + kBlk - 1) / kBlk;
  const bool in_place = p.base == p.y;
  const uint8_t* ws = p.ws + tile * tile_bytes(kTerms, p.v_ld);
  const uint16_t* vt = reinterpret_cast<const uint16_t*>(ws + sizeof(TileInfo));
  const uint32_t bar = smem_u32(s_bar);
  pdl_wait();
  if (tid == 0) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(bar));
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(bar + 8));
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    s_gave_up = 0;
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&s_tmem)),
                 "r"(kExpandCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid < static_cast<int>(sizeof(TileInfo) / 16))
    reinterpret_cast<uint4*>(&s_info)[tid] = reinterpret_cast<const uint4*>(ws)[tid];
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const int n_segments = s_info.n_segments;

  // The copies of B run ahead, with their own place: one 16-byte piece of
  // every 32nd row.  Order: groups, blocks of 128 rows, segments, 64 ranks.
  int l_g0 = 0, l_seg = 0, l_blk = 0, l_step = 0, l_stage = 0;
  const int l_pc = tid & 7;
  const int64_t l_at = static_cast<int64_t>(tid >> 3) * p.r_max + 8 * l_pc;
  const uint32_t l_off = operand_off(tid >> 3, l_pc);
  auto issue = [&]() {
    if (l_seg < n_segments) {
      const Piece sg = s_info.segment[l_seg];
      const int left = rows - l_blk * kBlk;  // rows of W from this block on
      const int rank = sg.rank - l_step * 64;
      const int pieces = min((rank + 15) / 16 * 2, 8);  // 16-byte pieces of whole MMA steps
      const uint16_t* b = p.b + (static_cast<int64_t>(max(sg.adapter, 0)) * p.rows + first +
                                 l_blk * kBlk) * p.r_max + l_step * 64;
      const uint32_t dst = st0 + l_stage * kBTile;
      if constexpr (VEC) {
        const int bytes = min(max(2 * (rank - 8 * l_pc), 0), 16);
        const int rows_in = min(left - (tid >> 3), kBlk);  // every 32nd of them
        const uint16_t* src = b + l_at;
        if (l_pc < pieces)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int n = 32 * i < rows_in ? bytes : 0;
            cp_async16(sm + dst + l_off + i * 4096, n ? src + i * 32ll * p.r_max : p.b, n);
          }
      } else if (pieces > 0) {
#pragma unroll 4
        for (int i = tid; i < kBlk * pieces * 8; i += kAdThreads) {
          const int row = i / (pieces * 8), k = i % (pieces * 8);
          uint16_t v = 0;
          if (k < rank && row < left) v = b[static_cast<int64_t>(row) * p.r_max + k];
          *reinterpret_cast<uint16_t*>(smp + dst + operand_off(row, k >> 3) + (k & 7) * 2) = v;
        }
      }
      l_stage = l_stage + 1 == STAGES ? 0 : l_stage + 1;
      if (NC > 1 && (l_step + 1) * 64 < sg.rank) {
        ++l_step;
      } else {
        l_step = 0;
        if (++l_seg == min(l_g0 + kGroup, n_segments)) {
          if (++l_blk == nb)
            l_blk = 0, l_g0 = l_seg;
          else
            l_seg = l_g0;
        }
      }
    }
    __syncwarp();
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) issue();

  // This thread's row within a block of 128, and its 32 tokens of the group.
  const int my_row = (warp & 3) * 32 + lane, n0 = (warp >> 2) * 32;
  const uint32_t t_addr = tmem + (static_cast<uint32_t>(warp & 3) * 32 << 16) + n0;
  int stage = 0;
  uint32_t phase = 0;
  for (int g0 = 0; g0 < n_segments; g0 += kGroup) {
    const int g1 = min(g0 + kGroup, n_segments);
    const int start = s_info.segment[g0].start;
    const int len = s_info.segment[g1 - 1].start + s_info.segment[g1 - 1].len - start;
    int r_all = 0;
    for (int i = g0; i < g1; ++i) r_all = max(r_all, s_info.segment[i].rank);
    const bool write = r_all > 0 || !in_place;
    // v's rows and the tokens' offsets; every thread is past the last group's
    // products and rows
    __syncthreads();
    const int pieces = (r_all + 15) / 16 * 2;
    if (tid >> 2 < len) {  // four threads a row
      const int row = tid >> 2;
      const uint16_t* src = vt + (start + row) * p.v_ld + 8 * (tid & 3);
      for (int c = 0; c < NC && 8 * c < pieces; ++c) {
        uint4 v[kTerms][2];
#pragma unroll
        for (int t = 0; t < kTerms; ++t)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (8 * c + (tid & 3) + 4 * i < pieces)
              v[t][i] = *reinterpret_cast<const uint4*>(src + t * kTileTokens * p.v_ld + 64 * c + 32 * i);
#pragma unroll
        for (int t = 0; t < kTerms; ++t)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (8 * c + (tid & 3) + 4 * i < pieces)
              *reinterpret_cast<uint4*>(smp + (t * NC + c) * kVTile +
                                        operand_off(row, (tid & 3) + 4 * i)) = v[t][i];
      }
    }
    if (tid < len) {
      s_base[tid] = s_info.tok[start + tid] * p.base_ld * static_cast<int64_t>(sizeof(E));
      s_y[tid] = s_info.tok[start + tid] * p.y_ld * static_cast<int64_t>(sizeof(E));
    }
    __syncthreads();
    const int n_tok = min(max(len - n0, 0), 32);
    // 32 whole neighbours: their rows are one stride apart
    bool run = n_tok == 32;
    if (run) {
      const int t = s_info.tok[start + n0 + lane];
      run = __all_sync(0xffffffffu, t == __shfl_sync(0xffffffffu, t, 0) + lane);
    }
    const int64_t base_step = p.base_ld * static_cast<int64_t>(sizeof(E)),
                  y_step = p.y_ld * static_cast<int64_t>(sizeof(E));
    const uint32_t idesc = mma_idesc((len + 15) / 16 * 16);
    E add[32];  // base of this thread's row
    const uint8_t* base = reinterpret_cast<const uint8_t*>(static_cast<const E*>(p.base) + first + my_row);
    uint8_t* y = reinterpret_cast<uint8_t*>(static_cast<E*>(p.y) + first + my_row);
    auto load_base = [&](int blk) {
      if (!p.base || !write || blk * kBlk + my_row >= rows) return;
      const uint8_t* src = base + blk * kBlk * static_cast<int>(sizeof(E));
      if (run) {
        src += s_base[n0];
#pragma unroll
        for (int j = 0; j < 32; ++j, src += base_step) add[j] = *reinterpret_cast<const E*>(src);
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (j < n_tok) add[j] = *reinterpret_cast<const E*>(src + s_base[n0 + j]);
      }
    };
    // the next block's base on its way to the L2 before its loads, a lane a token:
    // one instruction asks for the warp's 32 lines, and no register waits for them
    // (copying alone 113 -> 93 us at 4096 tokens x 14336 rows; two blocks ahead
    // 90, three 100, five 116)
    auto prefetch_base = [&](int blk) {
      const int c = blk * kBlk + (warp & 3) * 32;
      if (p.base && write && lane < n_tok && c < rows)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(
            reinterpret_cast<const uint8_t*>(static_cast<const E*>(p.base) + first + c) +
            s_base[n0 + lane]));
    };
#pragma unroll
    for (int j = 0; j < 32; ++j) add[j] = E(0);
    load_base(0);
    for (int blk = 0; blk < nb; ++blk) {
      prefetch_base(blk + 1);
      for (int seg = g0; seg < g1; ++seg) {
        const int rank = s_info.segment[seg].rank;
        for (int r0 = 0; r0 == 0 || (NC > 1 && r0 < rank); r0 += 64) {
          asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncthreads();  // this step's B is there, the accumulators have been read
          const int n_k = min((rank - r0 + 15) / 16, 4);  // MMA steps of a term
          if (warp == 0 && n_k > 0 && -2 - p.stall_tile != tile) {
            tc_fence_after();
            if (elect_one()) {
              const uint64_t b = operand_desc(sm + st0 + stage * kBTile);
              const uint32_t d = tmem + (seg - g0) * 64;
#pragma unroll
              for (int t = kTerms - 1; t >= 0; --t) {  // small terms first: fewer sums cut off
                const uint64_t v = operand_desc(sm + (t * NC + (r0 >> 6)) * kVTile);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  if (k < n_k)
                    tc_mma(d, b + 2 * k, v + 2 * k, idesc, (NC > 1 ? r0 : 0) | (kTerms - 1 - t) | k);
              }
              asm volatile(
                  "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                      bar)
                  : "memory");
            }
            __syncwarp();
          }
          stage = stage + 1 == STAGES ? 0 : stage + 1;
          issue();  // into the stage of the step before, whose products are done
          if (n_k > 0) {
            mbar_wait(bar, phase, &s_gave_up, p.wait_ns);
            phase ^= 1;
          }
        }
      }
      // base plus the token's own segment's column, 16 tokens at a time
      float v[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        if constexpr (F32)
          v[j] = add[j];
        else
          v[j] = bf16_value(add[j]);
      }
      if (blk + 1 < nb) load_base(blk + 1);
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        for (int seg = g0; seg < g1; ++seg) {  // the same for the warp
          const int from = s_info.segment[seg].start - start - n0 - 16 * c;
          const int to = from + s_info.segment[seg].len;
          if (s_info.segment[seg].rank == 0 || from >= 16 || to <= 0) continue;
          float d[16];
          tmem_ld16(t_addr + (seg - g0) * 64 + 16 * c, d);
          if (from <= 0 && to >= 16) {
#pragma unroll
            for (int j = 0; j < 16; ++j) v[16 * c + j] += d[j];
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (j >= from && j < to) v[16 * c + j] += d[j];
          }
        }
      }
      tc_fence_before();
      if (write && blk * kBlk + my_row < rows) {
        uint8_t* dst = y + blk * kBlk * static_cast<int>(sizeof(E));
        auto put = [&](uint8_t* at, float f) {
          if constexpr (F32)
            *reinterpret_cast<float*>(at) = f;
          else
            *reinterpret_cast<uint16_t*>(at) = bf16_bits(f);
        };
        if (run) {
          dst += s_y[n0];
#pragma unroll
          for (int j = 0; j < 32; ++j, dst += y_step) put(dst, v[j]);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (j < n_tok) put(dst + s_y[n0 + j], v[j]);
        }
      }
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  if (s_gave_up) {  // NaN over what this block has written for tokens with an adapter
    for (int i = 0; i < n_segments; ++i) {
      const Piece sg = s_info.segment[i];
      if (sg.rank == 0) continue;
      for (int t = sg.start; t < sg.start + sg.len; ++t)
        for (int r = tid; r < rows; r += kAdThreads) {
          E* at = static_cast<E*>(p.y) + s_info.tok[t] * p.y_ld + first + r;
          if constexpr (F32)
            *at = lost_value();
          else
            *at = bf16_bits(lost_value());
        }
    }
    drain_products(bar + 8, p.wait_ns);
  }
  tc_fence_after();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kExpandCols));
}

// ---- host ------------------------------------------------------------------

int env_int(const char* name, int otherwise) {
  const char* v = std::getenv(name);
  return v ? std::atoi(v) : otherwise;
}

// The kernel's dynamic shared memory limit, once per device.
template <auto kernel>
cudaError_t allow_smem(size_t bytes) {
  static std::mutex mu;
  static size_t allowed[kMaxDevices] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (allowed[dev] >= bytes) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(bytes));
  if (e == cudaSuccess) allowed[dev] = bytes;
  return e;
}

template <typename K>
cudaError_t launch(K* kernel, int64_t grid, int cluster, size_t smem, cudaStream_t s,
                   const AdapterParams& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kAdThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// v's rows, in elements: whole 32-rank steps, 64 bytes modulo 128 apart, so
// that 8 lanes' 16-byte shared-memory loads of two rows take all banks
int v_stride(int max_rank) {
  const int r32 = (max_rank + 31) / 32 * 32;
  return r32 % 64 == 0 ? r32 + 32 : r32;
}

// Few tokens: one launch.
template <int NT, bool MULTI, bool F32, bool VEC>
cudaError_t launch_few(AdapterParams p, cudaStream_t s) {
  constexpr int kTile = 16 * 8 * NT;
  // a window holds at most one piece per 16 tokens and one more per adapter
  // or none at all
  const int64_t most = static_cast<int64_t>(p.n) + 1 + kWindow / 16;
  p.per_window = static_cast<int>(most < kWindow ? most : kWindow);
  const int full = p.T / kWindow, rest = p.T % kWindow;
  const int64_t last = static_cast<int64_t>(p.n) + 1 + rest / 16;
  const int64_t clusters = static_cast<int64_t>(full) * p.per_window + (last < rest ? last : rest);
  const size_t smem = sizeof(float) * kTile * (kAdWarps + (MULTI ? 2 : 1) * kAdCluster) +
                      sizeof(uint16_t) * p.n_terms * 16 * p.v_ld;
  const cudaError_t e = allow_smem<adapter_kernel<NT, MULTI, F32, VEC>>(smem);
  if (e != cudaSuccess) return e;
  return launch(adapter_kernel<NT, MULTI, F32, VEC>, clusters * kAdCluster, kAdCluster, smem, s, p);
}
template <bool F32, bool VEC>
cudaError_t launch_few(const AdapterParams& p, cudaStream_t s) {
  if (p.r_max <= 16) return launch_few<2, false, F32, VEC>(p, s);
  if (p.r_max <= 32) return launch_few<4, false, F32, VEC>(p, s);
  if (p.r_max <= 64) return launch_few<8, false, F32, VEC>(p, s);
  return launch_few<8, true, F32, VEC>(p, s);
}

// Many: two.
template <bool VEC>
cudaError_t launch_shrink(const AdapterParams& p, int64_t tiles, cudaStream_t s) {
  const size_t smem = 1024 + kShrinkStages * kShrinkStage;
  const cudaError_t e = allow_smem<shrink_kernel<VEC>>(smem);
  if (e != cudaSuccess) return e;
  return launch(shrink_kernel<VEC>, tiles * p.split, p.split, smem, s, p);
}
template <int NC, bool F32, bool VEC>
cudaError_t launch_expand(const AdapterParams& p, int64_t blocks, cudaStream_t s) {
  const size_t smem = 1024 + NC * (F32 ? 3 : 2) * kVTile + kExpandStages * kBTile;
  const cudaError_t e = allow_smem<expand_kernel<NC, F32, VEC>>(smem);
  if (e != cudaSuccess) return e;
  return launch(expand_kernel<NC, F32, VEC>, blocks, 1, smem, s, p);
}
template <bool F32, bool VEC>
cudaError_t launch_expand(const AdapterParams& p, int64_t blocks, cudaStream_t s) {
  return p.r_max <= 64 ? launch_expand<1, F32, VEC>(p, blocks, s)
                       : launch_expand<4, F32, VEC>(p, blocks, s);
}

bool aligned_to(const void* p, uintptr_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

}  // namespace
}  // namespace pw

extern "C" int64_t pw_adapters_workspace_bytes(int32_t T, int32_t max_rank, int32_t y_type) {
  if (T <= pw::kNarrow || max_rank < 1 || max_rank > PW_MAX_ADAPTER_RANK) return 0;
  const int64_t tiles = (static_cast<int64_t>(T) + pw::kTileTokens - 1) / pw::kTileTokens;
  return tiles * pw::tile_bytes(y_type == PW_F32 ? 3 : 2, pw::v_stride(max_rank));
}

extern "C" pw_status_t pw_adapters(const uint16_t* d_x, int64_t x_stride, const uint16_t* d_a,
                                   const uint16_t* d_b, const int32_t* d_ids,
                                   const int32_t* d_ranks, const float* d_scale,
                                   int32_t n_adapters, int32_t max_rank, int32_t T, int32_t cols,
                                   int32_t rows, const void* d_base, int64_t base_stride,
                                   void* d_y, int32_t y_type, int64_t y_stride,
                                   void* d_workspace, int64_t workspace_bytes,
                                   pw_stream_t stream) {
  using namespace pw;
  auto bad = [](const char* msg) { return record_error(PW_ERR_INVALID_ARG, msg); };
  if (T < 0 || cols < 1 || rows < 1) return bad("pw_adapters: need T >= 0, cols >= 1, rows >= 1");
  if (cols > (1 << 28) || rows > (1 << 28))
    return record_error(PW_ERR_UNSUPPORTED, "pw_adapters: cols or rows above 2^28");
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
  if (workspace_bytes < pw_adapters_workspace_bytes(T, max_rank, y_type) ||
      (pw_adapters_workspace_bytes(T, max_rank, y_type) > 0 &&
       (!d_workspace || !aligned_to(d_workspace, 16))))
    return bad("pw_adapters: the workspace is smaller than pw_adapters_workspace_bytes, or not 16-byte "
               "aligned");
  AdapterParams p{};
  p.ws = static_cast<uint8_t*>(d_workspace);
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
  // rows that are 16-byte aligned and whole 16-byte pieces: of x and A, of B,
  // of base and y
  const int64_t per16 = 16 / static_cast<int64_t>(size);
  const bool vec_x = cols % 8 == 0 && x_stride % 8 == 0 && aligned_to(d_x, 16) && aligned_to(d_a, 16);
  const bool vec_b = max_rank % 8 == 0 && aligned_to(d_b, 16);
  const bool vec_y = rows % per16 == 0 && y_stride % per16 == 0 && aligned_to(d_y, 16) &&
                     (!d_base || (base_stride % per16 == 0 && aligned_to(d_base, 16)));
  p.v_ld = v_stride(max_rank);
  p.r32 = (max_rank + 31) / 32 * 32;
  p.n_terms = y_type == PW_F32 ? 3 : 2;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int dev = 0, n_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return record_error(PW_ERR_CUDA, cudaGetErrorString(e));
  const bool f32 = y_type == PW_F32;
  const int64_t tiles = (static_cast<int64_t>(T) + kTileTokens - 1) / kTileTokens;
  const int n_blk = (rows + kBlk - 1) / kBlk;
  // rows of an expand tile, in 128s: the fewest steps over the rounds of blocks
  // the GPU takes (two blocks an SM, one above rank 64), a block's start
  // counted as two steps
  int64_t least = INT64_MAX;
  const int64_t slots = (max_rank <= 64 ? 2 : 1) * n_sm;
  for (int per = 1; per <= n_blk; ++per) {
    const int64_t n = tiles * ((n_blk + per - 1) / per);
    const int64_t steps = (n + slots - 1) / slots * (per + 2);
    if (steps < least) least = steps, p.tile_rows = per * kBlk;
    if (n <= slots) break;
  }
  const int64_t blocks = tiles * ((rows + p.tile_rows - 1) / p.tile_rows);
  if (T > kNarrow && blocks >= (1ll << 31))
    return record_error(PW_ERR_UNSUPPORTED, "pw_adapters: T * rows too large for one launch");
  if (T <= kNarrow) {
    const bool vec = vec_x && vec_b && vec_y;
    e = f32 ? (vec ? launch_few<true, true>(p, s) : launch_few<true, false>(p, s))
            : (vec ? launch_few<false, true>(p, s) : launch_few<false, false>(p, s));
  } else {
    // waits are limited to two seconds, or as the test switches say
    const int wait_us = env_int("PW_TEST_WAIT_US", 0);
    p.wait_ns = wait_us > 0 ? wait_us * 1000ull : 2000000000ull;
    p.stall_tile = env_int("PW_TEST_STALL_TILE", -1);
    // columns split while the blocks fit the GPU twice over
    p.split = kAdCluster;
    while (p.split > 1 && tiles * p.split > 2 * n_sm) p.split /= 2;
    e = vec_x ? launch_shrink<true>(p, tiles, s) : launch_shrink<false>(p, tiles, s);
    if (e != cudaSuccess) return record_error(PW_ERR_CUDA, cudaGetErrorString(e));
    e = f32 ? (vec_b ? launch_expand<true, true>(p, blocks, s) : launch_expand<true, false>(p, blocks, s))
            : (vec_b ? launch_expand<false, true>(p, blocks, s)
                     : launch_expand<false, false>(p, blocks, s));
  }
  if (e != cudaSuccess) return record_error(PW_ERR_CUDA, cudaGetErrorString(e));
  return PW_OK;
}
