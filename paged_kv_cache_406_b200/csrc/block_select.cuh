// Block bounds and block selection for block-sparse decode.
//
// bounds[block][kv head][0 / 1][D]: the smallest and the largest value of each
// key channel over the block's tokens, in the pool's type (a minimum is one of
// the values, so nothing is rounded).
//
// The score of block j for KV head g of a sequence is an upper bound of q.k
// over the block's keys k and the heads h of the group:
//     score = max_h sum_d ( min(q_hd, 0) lo_jd + max(q_hd, 0) hi_jd ).
// The first n_first and last n_last blocks and the best of the others are
// selected; the ranking is that of exact arithmetic (ties to the lower index):
// score_kernel computes 32-bit scores with a bound of their error, and
// select_kernel scores the blocks near the border again in 64 bits.
#pragma once

#include <cuda_fp8.h>

#include "decode.cuh"
#include "device_common.cuh"
#include "rope.cuh"

namespace pkv {

// e4m3 pools are named by this element type.
struct E4m3 {
  uint8_t code;
};

// ---------------------------------------------------------------------------
// bounds: one warp per (sequence, touched block, KV head).  Bytes bound it:
// every row of a touched block is read once.  A row is D * sizeof(T) / 16
// lanes wide; the warp's lane groups take the rows in turn, each lane keeps
// the minimum and maximum of its 16 bytes, and the groups join by shuffles.
// ---------------------------------------------------------------------------
struct BoundsArgs {
  const void* k_pool;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  const int32_t* new_tokens;  // NULL: one per sequence
  void* bounds;
  int32_t num_seqs, num_blocks, num_kv_heads, max_blocks, block_size;
  int32_t max_new, window;  // window: blocks that max_new tokens can touch
};

template <typename T>
struct MinMax;

template <>
struct MinMax<float> {
  static constexpr int kRegs = 4;
  using Reg = float;
  __device__ static Reg mn(Reg a, Reg b) {
    Reg r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
  }
  __device__ static Reg mx(Reg a, Reg b) {
    Reg r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
  }
  __device__ static void load(const uint4& c, Reg (&x)[kRegs]) {
    x[0] = __uint_as_float(c.x);
    x[1] = __uint_as_float(c.y);
    x[2] = __uint_as_float(c.z);
    x[3] = __uint_as_float(c.w);
  }
  __device__ static uint4 store(const Reg (&x)[kRegs]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
  __device__ static Reg shfl(Reg x, int o) { return __shfl_xor_sync(kFull, x, o); }
};

template <typename V2>
struct MinMax16 {
  static constexpr int kRegs = 4;
  using Reg = V2;
  __device__ static Reg mn(Reg a, Reg b) { return __hmin2_nan(a, b); }
  __device__ static Reg mx(Reg a, Reg b) { return __hmax2_nan(a, b); }
  __device__ static Reg as(uint32_t w) { return *reinterpret_cast<const V2*>(&w); }
  __device__ static uint32_t bits(Reg x) { return *reinterpret_cast<const uint32_t*>(&x); }
  __device__ static void load(const uint4& c, Reg (&x)[kRegs]) {
    x[0] = as(c.x);
    x[1] = as(c.y);
    x[2] = as(c.z);
    x[3] = as(c.w);
  }
  __device__ static uint4 store(const Reg (&x)[kRegs]) { return make_uint4(bits(x[0]), bits(x[1]), bits(x[2]), bits(x[3])); }
  __device__ static Reg shfl(Reg x, int o) { return as(__shfl_xor_sync(kFull, bits(x), o)); }
};
template <>
struct MinMax<__nv_bfloat16> : MinMax16<__nv_bfloat162> {};
template <>
struct MinMax<__half> : MinMax16<__half2> {};

// Two e4m3 codes (low 16 bits) as a pair of f16 values, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes & 0xffffu), __NV_E4M3);
  return static_cast<uint32_t>(h.x) | (static_cast<uint32_t>(h.y) << 16);
}

// Codes are compared as the f16 values they stand for; converting a minimum
// back to e4m3 is exact.
template <>
struct MinMax<E4m3> {
  static constexpr int kRegs = 8;
  using Reg = __half2;
  using M = MinMax16<__half2>;
  __device__ static Reg mn(Reg a, Reg b) { return __hmin2_nan(a, b); }
  __device__ static Reg mx(Reg a, Reg b) { return __hmax2_nan(a, b); }
  __device__ static void load(const uint4& c, Reg (&x)[kRegs]) {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = M::as(e4m3x2_to_f16x2(w[i]));
      x[2 * i + 1] = M::as(e4m3x2_to_f16x2(w[i] >> 16));
    }
  }
  __device__ static uint4 store(const Reg (&x)[kRegs]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(x[2 * i]), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(x[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
      w[i] = lo | (hi << 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ static Reg shfl(Reg x, int o) { return M::shfl(x, o); }
};

template <typename T, int D>
__global__ void __launch_bounds__(256) block_bounds_kernel(const BoundsArgs a) {
  using MM = MinMax<T>;
  constexpr int kLanes = D * sizeof(T) / 16;  // lanes of a row
  constexpr int kGroups = 32 / kLanes;        // rows read at a time
  constexpr int kMaxRows = 32 / kGroups;      // rows of a lane in the largest block
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t w = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const int h = static_cast<int>(w % a.num_kv_heads);
  const int64_t bj = w / a.num_kv_heads;
  const int b = static_cast<int>(bj / a.window), i = static_cast<int>(bj % a.window);
  if (b >= a.num_seqs) return;
  const int bs = a.block_size;
  const int L = a.seq_lens[b], n = a.new_tokens ? a.new_tokens[b] : min(1, L);
  if (L < 0 || L > a.max_blocks * bs || n < 0 || n > L || n > a.max_new) {
    if (i == 0 && h == 0 && lane == 0) record_error(PKV_ERR_INVALID_ARG);
    return;
  }
  if (n == 0) return;
  const int j = (L - n) / bs + i;
  const int fill = min(bs, L - j * bs);
  if (fill <= 0) return;
  const int phys = a.block_tables[static_cast<int64_t>(b) * a.max_blocks + j];
  if (static_cast<unsigned>(phys) >= static_cast<unsigned>(a.num_blocks)) {
    if (h == 0 && lane == 0) record_error(PKV_ERR_BAD_BLOCK);
    return;
  }
  const int64_t tile = static_cast<int64_t>(phys) * a.num_kv_heads + h;
  const uint4* src = static_cast<const uint4*>(a.k_pool) + tile * bs * kLanes + lane;
  const int group = lane / kLanes;
  typename MM::Reg lo[MM::kRegs], hi[MM::kRegs];
  // every lane group reads a valid row first: row `group`, or row 0 of a
  // shorter block (a repeated row changes neither minimum nor maximum)
  {
    const uint4 c = src[group < fill ? 0 : -static_cast<int64_t>(group) * kLanes];
    MM::load(c, lo);
    MM::load(c, hi);
  }
#pragma unroll
  for (int r = 1; r < kMaxRows; ++r) {
    if (r * kGroups + group < fill) {
      typename MM::Reg x[MM::kRegs];
      MM::load(src[r * 32], x);
#pragma unroll
      for (int k = 0; k < MM::kRegs; ++k) {
        lo[k] = MM::mn(lo[k], x[k]);
        hi[k] = MM::mx(hi[k], x[k]);
      }
    }
  }
#pragma unroll
  for (int o = kLanes; o < 32; o <<= 1) {
#pragma unroll
    for (int k = 0; k < MM::kRegs; ++k) {
      lo[k] = MM::mn(lo[k], MM::shfl(lo[k], o));
      hi[k] = MM::mx(hi[k], MM::shfl(hi[k], o));
    }
  }
  uint4* dst = static_cast<uint4*>(a.bounds) + tile * 2 * kLanes + lane;
  if (lane < kLanes) {
    dst[0] = MM::store(lo);
    dst[kLanes] = MM::store(hi);
  }
}

// ---------------------------------------------------------------------------
// scores in 32 bits
// ---------------------------------------------------------------------------
struct SelectArgs {
  const void* q;       // dtype[num_seqs][num_q_heads][D]; f16 for e4m3 bounds
  const void* bounds;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  float* scores;       // [num_seqs * num_kv_heads][width]
  float* chunk_max;    // [num_seqs * num_kv_heads][chunks]: largest |bound| of a chunk
  double* fine;        // [num_seqs * num_kv_heads][width]: 64-bit scores, where there are too many for shared memory
  int32_t* selected;   // [num_seqs][num_kv_heads][max_selected]
  int32_t num_seqs, num_q_heads, num_kv_heads, num_blocks, max_blocks, block_size;
  int32_t max_selected, n_first, n_last;
  int32_t width, chunks;
};

constexpr int kScoreThreads = 256;
constexpr int kScoreChunk = 256;  // blocks of one CTA

// Blocks of sequence b (0 for a length outside the table's capacity, which is
// recorded).
__device__ __forceinline__ int blocks_of(const SelectArgs& a, int b, bool record) {
  const int L = a.seq_lens[b];
  if (L < 0 || L > a.max_blocks * a.block_size) {
    if (record) record_error(PKV_ERR_INVALID_ARG);
    return 0;
  }
  return (L + a.block_size - 1) / a.block_size;
}

__device__ __forceinline__ int64_t bounds_tile(const SelectArgs& a, int b, int j, int g) {
  int phys = a.block_tables[static_cast<int64_t>(b) * a.max_blocks + j];
  if (static_cast<unsigned>(phys) >= static_cast<unsigned>(a.num_blocks)) {
    record_error(PKV_ERR_BAD_BLOCK);
    phys = 0;
  }
  return static_cast<int64_t>(phys) * a.num_kv_heads + g;
}

// The type q comes in for bounds of type T.
template <typename T>
struct QueryOf { using type = T; };
template <>
struct QueryOf<E4m3> { using type = __half; };

// Element d of a bounds row as a float.
template <typename T>
__device__ __forceinline__ float bound_at(const void* base, int64_t i) {
  if constexpr (std::is_same_v<T, E4m3>) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<const uint8_t*>(base)[i], __NV_E4M3);
    return __half2float(__half(h));
  } else {
    return widen1<T>(static_cast<const T*>(base)[i]);
  }
}

// One warp per block, lanes over the channels.  Bytes bound it: 2 D elements
// per block and KV head are read once for the G heads of the group.
template <typename T, int D, int G>
__global__ void __launch_bounds__(kScoreThreads) score_kernel(const SelectArgs a) {
  using Q = typename QueryOf<T>::type;
  constexpr int kPer = D / 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int row = blockIdx.x / a.chunks, chunk = blockIdx.x - row * a.chunks;
  const int b = row / a.num_kv_heads, g = row - b * a.num_kv_heads;
  const int nblk = blocks_of(a, b, chunk == 0 && g == 0 && threadIdx.x == 0);
  const int j0 = chunk * kScoreChunk;
  if (nblk <= a.max_selected || j0 >= nblk) return;  // every block is selected, or none is here
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float neg[G][kPer], pos[G][kPer];
#pragma unroll
  for (int h = 0; h < G; ++h)
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const float x = widen1<Q>(static_cast<const Q*>(a.q)[(static_cast<int64_t>(b) * a.num_q_heads + g * G + h) * D + i * 32 + lane]);
      neg[h][i] = x < 0.f ? x : (x == x ? 0.f : x);
      pos[h][i] = x > 0.f ? x : (x == x ? 0.f : x);
    }
  float big = 0.f;
  const int j1 = min(nblk, j0 + kScoreChunk);
  for (int j = j0 + warp; j < j1; j += kScoreThreads / 32) {
    const int64_t at = bounds_tile(a, b, j, g) * 2 * D + lane;
    float s[G];
#pragma unroll
    for (int h = 0; h < G; ++h) s[h] = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const float lo = bound_at<T>(a.bounds, at + i * 32), hi = bound_at<T>(a.bounds, at + D + i * 32);
      big = MinMax<float>::mx(big, MinMax<float>::mx(fabsf(lo), fabsf(hi)));
#pragma unroll
      for (int h = 0; h < G; ++h) s[h] += neg[h][i] * lo + pos[h][i] * hi;
    }
    float best = 0.f;
#pragma unroll
    for (int h = 0; h < G; ++h) {
#pragma unroll
      for (int o = 16; o; o >>= 1) s[h] += __shfl_xor_sync(kFull, s[h], o);
      best = h ? MinMax<float>::mx(best, s[h]) : s[0];
    }
    if (lane == 0) a.scores[static_cast<int64_t>(row) * a.width + j] = best;
  }
  __shared__ float red[kScoreThreads / 32];
#pragma unroll
  for (int o = 16; o; o >>= 1) big = MinMax<float>::mx(big, __shfl_xor_sync(kFull, big, o));
  if (lane == 0) red[warp] = big;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kScoreThreads / 32; ++w) big = MinMax<float>::mx(big, red[w]);
    a.chunk_max[static_cast<int64_t>(row) * a.chunks + chunk] = big;
  }
}

// ---------------------------------------------------------------------------
// the selection: one CTA per (sequence, KV head)
// ---------------------------------------------------------------------------
constexpr int kSelectThreads = 512;
constexpr int kSelectBins = 2048;
constexpr int kSelectFine = 512;  // border blocks ranked in shared memory

// Error bound of a 32-bit score over sum_d |q_d| times the largest |bound|.
// The longest chain of sums is 2 D = 256 products: in 32-bit adds it loses at
// most 256 x 2^-24 = 2^-16 of that.  Tensor cores align the 16 products and
// the sum of a step to the largest of them and drop bits below 2^-23 of it:
// 17 x 2^-23 a step, 16 steps, 2^-14.9.
constexpr float kScoreError = 1.0f / 16384;

// Order-preserving map of floats to unsigned integers; NaN above everything.
__device__ __forceinline__ uint32_t key32(float x) {
  if (x != x) return 0xffffffffu;
  x += 0.0f;  // -0 and 0 are equal
  const uint32_t u = __float_as_uint(x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unkey32(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ uint64_t key64(double x) {
  if (x != x) return ~0ull;
  x += 0.0;
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(x));
  return u >> 63 ? ~u : u | (1ull << 63);
}

// The score of block j in 64 bits (all lanes of the warp get it).
template <typename T, int D>
__device__ __forceinline__ uint64_t fine_key(const SelectArgs& a, int b, int g, int G, int j) {
  using Q = typename QueryOf<T>::type;
  const int lane = threadIdx.x & 31;
  const int64_t at = bounds_tile(a, b, j, g) * 2 * D + lane;
  double lo[D / 32], hi[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    lo[i] = bound_at<T>(a.bounds, at + i * 32);
    hi[i] = bound_at<T>(a.bounds, at + D + i * 32);
  }
  uint64_t best = 0;
#pragma unroll 1
  for (int h = 0; h < G; ++h) {
    double s = 0;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const float x = widen1<Q>(static_cast<const Q*>(a.q)[(static_cast<int64_t>(b) * a.num_q_heads + g * G + h) * D + i * 32 + lane]);
      const double xn = x > 0.f ? 0.0 : x, xp = x < 0.f ? 0.0 : x;
      s += xn * lo[i] + xp * hi[i];
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
    const uint64_t k = key64(s);
    best = k > best ? k : best;
  }
  return best;
}

// Block-wide sum of one value per thread; `red` holds a word per warp.
__device__ __forceinline__ int block_sum(int x, int* red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  int s = 0;
  for (int w = 0; w < kSelectThreads / 32; ++w) s += red[w];
  return s;
}

// Finds in hist[0 .. bins) (counts per bin, larger keys in higher bins) the
// bin in which the need-th largest lies: returns it, and in *above the count
// in higher bins.
__device__ __forceinline__ int find_bin(const int* hist, int bins, int need, int* above, int* red, int* shared2) {
  // thread t owns bins - 1 - t * per ... downwards
  const int per = (bins + kSelectThreads - 1) / kSelectThreads;
  int mine = 0;
  const int top = bins - 1 - static_cast<int>(threadIdx.x) * per;
  for (int i = 0; i < per; ++i)
    if (top - i >= 0) mine += hist[top - i];
  int before = mine;  // inclusive prefix over the warp
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, before, o);
    if (lane >= o) before += y;
  }
  __syncthreads();
  if (lane == 31) red[warp] = before;
  __syncthreads();
  for (int w = 0; w < warp; ++w) before += red[w];
  before -= mine;  // exclusive
  if (before < need && before + mine >= need) {
    int run = before;
    for (int i = 0; i < per; ++i) {
      const int k = top - i;
      if (k < 0) break;
      if (run + hist[k] >= need) {
        shared2[0] = k;
        shared2[1] = run;
        break;
      }
      run += hist[k];
    }
  }
  __syncthreads();
  *above = shared2[1];
  return shared2[0];
}

template <typename T, int D>
__global__ void __launch_bounds__(kSelectThreads) select_kernel(const SelectArgs a) {
  using Q = typename QueryOf<T>::type;
  extern __shared__ uint32_t bitmap[];  // one bit per block
  __shared__ int hist[kSelectBins];
  __shared__ uint64_t fine[kSelectFine];
  __shared__ int fine_at[kSelectFine];
  __shared__ int red[kSelectThreads / 32], two[2], count;
  __shared__ uint32_t range[2];
  __shared__ float eps_s;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int g = blockIdx.x % a.num_kv_heads, b = blockIdx.x / a.num_kv_heads;
  const int G = a.num_q_heads / a.num_kv_heads;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t row = blockIdx.x;
  const int nblk = blocks_of(a, b, false);
  const int K = a.max_selected;
  int32_t* out = a.selected + row * K;
  if (nblk <= K) {
    for (int i = tid; i < K; i += kSelectThreads) out[i] = i < nblk ? i : -1;
    return;
  }
  const int c0 = a.n_first, c1 = nblk - a.n_last;  // candidates [c0, c1): more than are needed, since nblk > K
  const int need0 = K - a.n_first - a.n_last;
  const int words = (nblk + 31) / 32;
  for (int i = tid; i < words; i += kSelectThreads) {
    uint32_t m = 0;
    for (int t = 0; t < 32; ++t) {
      const int j = i * 32 + t;
      if (j < nblk && (j < c0 || j >= c1)) m |= 1u << t;
    }
    bitmap[i] = m;
  }
  const float* scores = a.scores + row * a.width;

  if (need0 > 0) {
    // ---- the error bound of this row's scores ----
    if (warp == 0) {
      float q1 = 0.f;
      for (int h = 0; h < G; ++h) {
        float s = 0.f;
        for (int d = lane; d < D; d += 32)
          s += fabsf(widen1<Q>(static_cast<const Q*>(a.q)[(static_cast<int64_t>(b) * a.num_q_heads + g * G + h) * D + d]));
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
        q1 = MinMax<float>::mx(q1, s);
      }
      float big = 0.f;
      for (int i = lane; i < (nblk + kScoreChunk - 1) / kScoreChunk; i += 32)
        big = MinMax<float>::mx(big, a.chunk_max[row * a.chunks + i]);
#pragma unroll
      for (int o = 16; o; o >>= 1) big = MinMax<float>::mx(big, __shfl_xor_sync(kFull, big, o));
      if (lane == 0) eps_s = q1 * big * kScoreError;
    }
    if (tid == 0) {
      range[0] = 0xffffffffu;
      range[1] = 0;
    }
    __syncthreads();
    const float eps = eps_s;
    const bool bounded = eps <= 1e30f;  // false for infinities and NaN: every candidate is scored in 64 bits

    // ---- narrow the keys' range to a bin that holds the need0-th largest ----
    float t_lo = -INFINITY, t_hi = INFINITY;  // the need0-th largest score lies in [t_lo, t_hi]
    if (bounded) {
      uint32_t mn = 0xffffffffu, mx = 0;
      for (int j = c0 + tid; j < c1; j += kSelectThreads) {
        const uint32_t k = key32(scores[j]);
        mn = min(mn, k);
        mx = max(mx, k);
      }
      mn = __reduce_min_sync(kFull, mn);
      mx = __reduce_max_sync(kFull, mx);
      if (lane == 0) {
        atomicMin(&range[0], mn);
        atomicMax(&range[1], mx);
      }
      __syncthreads();
      uint32_t base = range[0], last = range[1];
      int need = need0;
      for (;;) {
        int shift = 0;
        while (((last - base) >> shift) >= kSelectBins) ++shift;
        for (int i = tid; i < kSelectBins; i += kSelectThreads) hist[i] = 0;
        __syncthreads();
        for (int j = c0 + tid; j < c1; j += kSelectThreads) {
          const uint32_t k = key32(scores[j]);
          if (k >= base && k <= last) atomicAdd(&hist[(k - base) >> shift], 1);
        }
        __syncthreads();
        int above;
        const int bin = find_bin(hist, kSelectBins, need, &above, red, two);
        const int in_bin = hist[bin];
        need -= above;
        const uint32_t nb = base + (static_cast<uint32_t>(bin) << shift);
        const uint32_t width = shift ? (1u << shift) - 1 : 0;
        last = last - nb < width ? last : nb + width;
        base = nb;
        __syncthreads();
        if (shift == 0 || in_bin <= 32) break;
      }
      t_lo = unkey32(base);
      t_hi = unkey32(last);
    }

    // ---- blocks surely in, and those near the border ----
    // exact scores are within eps of these: above t_hi + 2 eps a block beats
    // the border, below t_lo - 2 eps it does not reach it
    const float in_above = bounded ? t_hi + 2.f * eps : INFINITY;
    const float out_below = bounded ? t_lo - 2.f * eps : -INFINITY;
    if (tid == 0) count = 0;
    __syncthreads();
    int sure = 0;
    for (int j0 = 0; j0 < words * 32; j0 += kSelectThreads) {
      const int j = j0 + tid;
      bool in = false, near = false;
      if (j >= c0 && j < c1) {
        const float s = scores[j];
        in = bounded && s > in_above;
        near = !in && !(bounded && s < out_below);
      }
      const uint32_t m = __ballot_sync(kFull, in);
      if (lane == 0 && m) bitmap[j >> 5] |= m;
      sure += in;
      if (near) {
        const int at = atomicAdd(&count, 1);
        if (at < kSelectFine) fine_at[at] = j;
      }
    }
    sure = block_sum(sure, red);
    const int n_near = count;
    const int need = need0 - sure;  // of the near blocks

    if (n_near <= kSelectFine) {
      for (int i = warp; i < n_near; i += kSelectThreads / 32) {
        const uint64_t k = fine_key<T, D>(a, b, g, G, fine_at[i]);
        if (lane == 0) fine[i] = k;
      }
      __syncthreads();
      for (int i = tid; i < n_near; i += kSelectThreads) {
        const uint64_t k = fine[i];
        const int j = fine_at[i];
        int rank = 0;
        for (int x = 0; x < n_near; ++x) rank += fine[x] > k || (fine[x] == k && fine_at[x] < j);
        if (rank < need) atomicOr(&bitmap[j >> 5], 1u << (j & 31));
      }
    } else {
      // many blocks within the error of the border (equal keys, infinities):
      // 64-bit keys in global memory and a radix selection over them
      uint64_t* keys = reinterpret_cast<uint64_t*>(a.fine + row * a.width);
      for (int j = c0 + warp; j < c1; j += kSelectThreads / 32) {
        const float s = scores[j];
        const bool in = bounded && s > in_above;
        const bool near = !in && !(bounded && s < out_below);
        if (near) {
          const uint64_t k = fine_key<T, D>(a, b, g, G, j);
          if (lane == 0) keys[j] = k;
        }
      }
      __syncthreads();
      uint64_t prefix = 0;
      int left = need;
      for (int shift = 56; shift >= 0; shift -= 8) {
        for (int i = tid; i < 256; i += kSelectThreads) hist[i] = 0;
        __syncthreads();
        for (int j = c0 + tid; j < c1; j += kSelectThreads) {
          const float s = scores[j];
          if (bounded && (s > in_above || s < out_below)) continue;
          const uint64_t k = keys[j];
          if (shift == 56 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(k >> shift) & 255], 1);
        }
        __syncthreads();
        int above;
        const int bin = find_bin(hist, 256, left, &above, red, two);
        left -= above;
        prefix |= static_cast<uint64_t>(bin) << shift;
        __syncthreads();
      }
      // keys above `prefix`, and the first `left` equal to it
      int equal = 0;
      for (int j0 = 0; j0 < words * 32; j0 += kSelectThreads) {
        const int j = j0 + tid;
        bool in = false, eq = false;
        if (j >= c0 && j < c1) {
          const float s = scores[j];
          if (!(bounded && (s > in_above || s < out_below))) {
            in = keys[j] > prefix;
            eq = keys[j] == prefix;
          }
        }
        const uint32_t me = __ballot_sync(kFull, eq);
        __syncthreads();
        if (lane == 0) red[warp] = __popc(me);
        __syncthreads();
        int before = equal + __popc(me & ((1u << lane) - 1));
        for (int w = 0; w < kSelectThreads / 32; ++w) {
          if (w < warp) before += red[w];
          equal += red[w];
        }
        const uint32_t m = __ballot_sync(kFull, in || (eq && before < left));
        if (lane == 0 && m) bitmap[j >> 5] |= m;
      }
    }
  }
  __syncthreads();

  // ---- the bitmap as an ascending list ----
  int done = 0;
  for (int w0 = 0; w0 < words; w0 += kSelectThreads) {
    const int w = w0 + tid;
    uint32_t m = w < words ? bitmap[w] : 0;
    const int n = __popc(m);
    int at = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, at, o);
      if (lane >= o) at += y;
    }
    __syncthreads();
    if (lane == 31) red[warp] = at;
    __syncthreads();
    at += done - n;
    for (int x = 0; x < kSelectThreads / 32; ++x) {
      if (x < warp) at += red[x];
      done += red[x];
    }
    while (m) {
      if (at < K) out[at] = w * 32 + __ffs(m) - 1;
      ++at;
      m &= m - 1;
    }
  }
}

}  // namespace pkv
