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
// selected; the ranking is that of 64-bit sums (ties to the lower index):
// select_kernel computes 32-bit scores with a bound of their error and scores
// the blocks near the border again in 64 bits.
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
// the minimum and maximum of its 16 bytes, and the groups join by shuffles.  16
// prompts of up to 4096 f16 tokens (107 MB): 19 us, 5.6 TB/s; one block for
// each of 64 sequences: 2.3 us.
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
// selection: score_kernel, then select_kernel with one CTA per (sequence, KV
// head): 256 threads and four CTAs an SM, or 1024 threads for few long rows.
// Measured with the score kernel before the selection started under it, 256
// against 1024 threads: 16 rows of 8192 blocks 31 us against 24.5, 512 rows of
// 2048 blocks 71 against 99 (now 20.7 and 69.8 us).  The selection is a chain of short
// steps on one row (6 us for 512 blocks, 11 for 8192) and bound by their
// latency.  With eight heads of 128 it spills (up to 52 bytes stored and 148
// loaded a thread, in the 64-bit scores of the border).
// ---------------------------------------------------------------------------
struct TileStats {  // of 16 scores
  uint32_t min_key, max_key;  // the candidates' keys
  float big;                  // largest |bound|
  float pad;
};

struct SelectArgs {
  const void* q;       // dtype[num_seqs][num_q_heads][D]; f16 for e4m3 bounds
  const void* bounds;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  float* scores;       // [num_seqs * num_kv_heads][max_blocks]
  TileStats* stats;    // [num_seqs * num_kv_heads][tiles]
  uint64_t* fine;      // [num_seqs * num_kv_heads][max_blocks]: 64-bit keys, where there are too many for shared memory
  int32_t* selected;   // [num_seqs][num_kv_heads][max_selected]
  int32_t num_seqs, num_q_heads, num_kv_heads, num_blocks, max_blocks, block_size;
  int32_t max_selected, n_first, n_last;
  int32_t tiles;        // of 16 blocks, in max_blocks
  int32_t smem_scores;  // blocks whose scores fit the shared memory of the launch (0: re-read them)
  int32_t after_scores; // whether score_kernel is the launch before select_kernel
};

constexpr int kSelectBins = 1024;
constexpr int kSelectFine = 512;    // border blocks ranked in shared memory

// Error taken for a 32-bit score, over sum_d |q_d| times the largest |bound|.
// 32-bit sums of 2 D = 256 products lose at most 256 x 2^-24 = 2^-16 of that.
// How tensor cores sum is not documented; this assumes that they align the 16
// products and the sum of a step to the largest of them and drop bits below
// 2^-23 of it: 17 x 2^-23 a step, 16 steps, 2^-14.9.  Measured on sums that
// grow large and cancel, and on normal ones: 2^-24.7 at most.
// Products below 2^-126 may be lost altogether: 256 of them are below 1e-35.
constexpr float kScoreError = 1.0f / 16384, kScoreTiny = 1e-35f;

// Blocks of a sequence of length L (0 for a length outside the table's
// capacity, which is recorded).
__device__ __forceinline__ int blocks_of(const SelectArgs& a, int L, bool record) {
  if (L < 0 || L > a.max_blocks * a.block_size) {
    if (record) record_error(PKV_ERR_INVALID_ARG);
    return 0;
  }
  return (L + a.block_size - 1) / a.block_size;
}

// The tile (block, KV head) of a table entry.
__device__ __forceinline__ int64_t bounds_tile(const SelectArgs& a, int phys, int g) {
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

// A bound as a float.
template <typename T>
__device__ __forceinline__ float bound_value(T x) {
  if constexpr (std::is_same_v<T, E4m3>) return __half2float(__half(__nv_cvt_fp8_to_halfraw(x.code, __NV_E4M3)));
  else return widen1<T>(x);
}

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

// Scores of 16 blocks by one warp.  On the tensor cores the blocks are the 16
// rows of A, the heads the 8 columns of B and the 2 D bound channels the
// contraction, in an order of its own: each lane's 16-byte loads of a row are
// its A fragments as they come (channels e0 + 4 s .. + 3 of piece i in step
// s), and B is q in the same order, min(q, 0) against the minima and
// max(q, 0) against the maxima.
template <typename T, int D, int G>
struct Scorer {
  using Q = typename QueryOf<T>::type;
  using M = MinMax<Q>;
  static constexpr int kElems = 16 / static_cast<int>(sizeof(T));  // of a load
  static constexpr int kPieces = 2 * D / (4 * kElems);             // loads of a row by a lane
  static constexpr int kSteps = kElems / 4;                        // mma steps of a piece
  uint32_t q[kPieces][kSteps][2];
  uint4 x[2][kPieces];  // the tile's rows lane / 4 and lane / 4 + 8
  typename M::Reg big[4];

  __device__ __forceinline__ void group(const SelectArgs& a, int b, int g) {
    const int lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
    const typename M::Reg zero = M::as(0);
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int e0 = i * 4 * kElems + tq * kElems, d0 = e0 % D;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        uint2 w = make_uint2(0, 0);
        if (gq < G)
          w = *reinterpret_cast<const uint2*>(static_cast<const Q*>(a.q) +
                                              (static_cast<int64_t>(b) * a.num_q_heads + g * G + gq) * D + d0 + 4 * s);
        const typename M::Reg y0 = M::as(w.x), y1 = M::as(w.y);
        q[i][s][0] = M::bits(i < kPieces / 2 ? M::mn(y0, zero) : M::mx(y0, zero));
        q[i][s][1] = M::bits(i < kPieces / 2 ? M::mn(y1, zero) : M::mx(y1, zero));
      }
    }
  }

  // tile[r]: of row lane / 4 + 8 r
  __device__ __forceinline__ void load(const SelectArgs& a, const int64_t (&tile)[2]) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(a.bounds) + tile[r] * 2 * D) + (threadIdx.x & 3);
#pragma unroll
      for (int i = 0; i < kPieces; ++i) x[r][i] = __ldg(src + 4 * i);
    }
  }

  // The scores of the two rows (in all four lanes of a row), and the largest
  // |bound| this lane has met in the tile.
  __device__ __forceinline__ float2 score(float* largest) {
    const int tq = threadIdx.x & 3;
    // four chains for the maxima and two for the sums: one would wait for itself
    float c[2][4] = {};
#pragma unroll
    for (int k = 0; k < 4; ++k) big[k] = M::as(0);
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      uint32_t w[2][2 * kSteps];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint32_t v[4] = {x[r][i].x, x[r][i].y, x[r][i].z, x[r][i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if constexpr (sizeof(T) == 1) {
            w[r][2 * k] = e4m3x2_to_f16x2(v[k]);
            w[r][2 * k + 1] = e4m3x2_to_f16x2(v[k] >> 16);
          } else {
            w[r][k] = v[k];
          }
        }
#pragma unroll
        for (int k = 0; k < 2 * kSteps; ++k) big[k & 3] = M::mx(big[k & 3], __habs2(M::as(w[r][k])));
      }
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const uint32_t f[4] = {w[0][2 * s], w[1][2 * s], w[0][2 * s + 1], w[1][2 * s + 1]};
        mma_16816<Q>(c[s & 1], f, q[i][s][0], q[i][s][1]);
      }
    }
    using F = MinMax<float>;
    const bool h0 = 2 * tq < G, h1 = 2 * tq + 1 < G;
    float2 s = make_float2(h0 ? c[0][0] + c[1][0] : -INFINITY, h0 ? c[0][2] + c[1][2] : -INFINITY);
    if (h1) s = make_float2(F::mx(s.x, c[0][1] + c[1][1]), F::mx(s.y, c[0][3] + c[1][3]));
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      s.x = F::mx(s.x, __shfl_xor_sync(kFull, s.x, o));
      s.y = F::mx(s.y, __shfl_xor_sync(kFull, s.y, o));
    }
    Chunk<Q, 2> m;
    m.raw = M::bits(M::mx(M::mx(big[0], big[1]), M::mx(big[2], big[3])));
    *largest = F::mx(widen1<Q>(m.e[0]), widen1<Q>(m.e[1]));
    return s;
  }
};

// 32-bit bounds on the CUDA cores: lanes over the channels, four blocks at a
// time.
template <int D, int G>
struct Scorer<float, D, G> {
  static constexpr int kPieces = 2 * D / 128;
  float4 q[G][kPieces];
  int64_t now[2];
  const float* bounds;

  __device__ __forceinline__ void group(const SelectArgs& a, int b, int g) {
    using F = MinMax<float>;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int h = 0; h < G; ++h)
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int e0 = i * 128 + lane * 4;
        const float4 y = *reinterpret_cast<const float4*>(
            static_cast<const float*>(a.q) + (static_cast<int64_t>(b) * a.num_q_heads + g * G + h) * D + e0 % D);
        q[h][i] = e0 < D ? make_float4(F::mn(y.x, 0.f), F::mn(y.y, 0.f), F::mn(y.z, 0.f), F::mn(y.w, 0.f))
                         : make_float4(F::mx(y.x, 0.f), F::mx(y.y, 0.f), F::mx(y.z, 0.f), F::mx(y.w, 0.f));
      }
  }

  __device__ __forceinline__ void load(const SelectArgs& a, const int64_t (&tile)[2]) {
    bounds = static_cast<const float*>(a.bounds);
    now[0] = tile[0];
    now[1] = tile[1];
  }

  __device__ __forceinline__ float2 score(float* largest) {
    using F = MinMax<float>;
    const int lane = threadIdx.x & 31;
    float2 out = make_float2(0.f, 0.f);
    float big = 0.f;
#pragma unroll 1
    for (int r0 = 0; r0 < 16; r0 += 4) {
      float4 y[4][kPieces];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        // row r0 + r lies with lane 4 (row mod 8), in now[row / 8]
        const int64_t t = __shfl_sync(kFull, r0 < 8 ? now[0] : now[1], 4 * ((r0 + r) & 7));
        const float4* src = reinterpret_cast<const float4*>(bounds + t * 2 * D) + lane;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) y[r][i] = __ldg(src + 32 * i);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float best = 0.f;
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
          big = F::mx(big, F::mx(F::mx(fabsf(y[r][i].x), fabsf(y[r][i].y)), F::mx(fabsf(y[r][i].z), fabsf(y[r][i].w))));
#pragma unroll
        for (int h = 0; h < G; ++h) {
          float s = 0.f;
#pragma unroll
          for (int i = 0; i < kPieces; ++i)
            s += q[h][i].x * y[r][i].x + q[h][i].y * y[r][i].y + q[h][i].z * y[r][i].z + q[h][i].w * y[r][i].w;
#pragma unroll
          for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
          best = h ? F::mx(best, s) : s;
        }
        if ((lane >> 2) == ((r0 + r) & 7)) {
          if (r0 < 8) out.x = best;
          else out.y = best;
        }
      }
    }
    *largest = big;
    return out;
  }
};

// Bytes bound it: 2 D elements per block and KV head, read once for the G
// heads of the group.  The tiles of 16 blocks of all rows that have a choice
// to make are numbered in order and dealt out to the warps of a resident grid
// in equal runs, whatever the mix of lengths: a warp keeps q of its row in
// registers and streams the row's tiles.  64 contexts of 8K to 32K tokens (337
// MB of bf16 bounds): 58 us, 5.8 TB/s.  A CTA or a cluster per row took 79 to
// 97 us there (the longest row ends last); loads through shared memory
// (cp.async) 78, for the instructions around them.
constexpr int kScoreThreads = 256;
constexpr int kScoreWarps = kScoreThreads / 32;

template <typename T, int D, int G>
__global__ void __launch_bounds__(kScoreThreads, 2) score_kernel(const SelectArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gq = lane >> 2;
  // Every warp numbers the tiles by itself, 128 sequences (four a lane) at a
  // time; a short batch then waits for one trip to memory and no barrier.
  constexpr int kPer = 4;
  auto tiles_of = [&](int b) {
    const int nblk = b < a.num_seqs ? blocks_of(a, a.seq_lens[b], false) : 0;
    return nblk > a.max_selected ? (nblk + 15) / 16 : 0;
  };
  int count[kPer], mine = 0, total = 0;
  for (int b0 = (a.num_seqs - 1) / (32 * kPer) * (32 * kPer); b0 >= 0; b0 -= 32 * kPer) {  // ends with the first 128
    mine = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) mine += count[i] = tiles_of(b0 + lane * kPer + i);
    total += __reduce_add_sync(kFull, mine);
  }
  // neighbouring runs go to different SMs, so that a short list uses them all
  const int64_t w = static_cast<int64_t>(warp) * gridDim.x + blockIdx.x, nw = static_cast<int64_t>(gridDim.x) * kScoreWarps;
  const int64_t all = static_cast<int64_t>(total) * a.num_kv_heads;
  int64_t p = all * w / nw;
  const int64_t end = all * (w + 1) / nw;
  if (p >= end) return;
  int b = 0, first = 0;  // the sequence of tile p, and the tiles of a KV head before it
  for (int b0 = 0, done = 0;; b0 += 32 * kPer) {
    if (b0) {
      mine = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) mine += count[i] = tiles_of(b0 + lane * kPer + i);
    }
    int before = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, before, o);
      if (lane >= o) before += y;
    }
    const int sum = __shfl_sync(kFull, before, 31);
    before += done - mine;
    const bool here = static_cast<int64_t>(before) * a.num_kv_heads <= p && static_cast<int64_t>(before + mine) * a.num_kv_heads > p;
    const uint32_t m = __ballot_sync(kFull, here);
    if (m) {
      int at = b0 + lane * kPer;
#pragma unroll
      for (int i = 0; i < kPer - 1; ++i)
        if (at == b0 + lane * kPer + i && static_cast<int64_t>(before + count[i]) * a.num_kv_heads <= p) {
          before += count[i];
          ++at;
        }
      b = __shfl_sync(kFull, at, __ffs(m) - 1);
      first = __shfl_sync(kFull, before, __ffs(m) - 1);
      break;
    }
    done += sum;
  }
  int nblk = blocks_of(a, a.seq_lens[b], false), tiles = (nblk + 15) / 16;
  const int64_t off = p - static_cast<int64_t>(first) * a.num_kv_heads;
  int g = static_cast<int>(off / tiles), t = static_cast<int>(off - static_cast<int64_t>(g) * tiles);
  auto entry = [&](int r) {  // of row gq + 8 r of the tile at hand
    return a.block_tables[static_cast<int64_t>(b) * a.max_blocks + min(t * 16 + gq + 8 * r, nblk - 1)];
  };
  int32_t phys[2] = {entry(0), entry(1)};
  Scorer<T, D, G> scorer;
  scorer.group(a, b, g);
  for (;;) {
    const int64_t tile[2] = {bounds_tile(a, phys[0], g), bounds_tile(a, phys[1], g)};
    scorer.load(a, tile);
    const int64_t row = static_cast<int64_t>(b) * a.num_kv_heads + g;
    const int j0 = t * 16 + gq, c1 = nblk - a.n_last, blocks = nblk, at = t;
    // the tile after, and its table entries
    const bool more = ++p < end;
    bool other = false;
    if (more) {
      if (++t == tiles) {
        t = 0;
        other = true;
        if (++g == a.num_kv_heads) {
          g = 0;
          do tiles = tiles_of(++b);  // there is one: p < end
          while (tiles == 0);
          nblk = blocks_of(a, a.seq_lens[b], false);
        }
      }
      phys[0] = entry(0);
      phys[1] = entry(1);
    }
    float big;
    const float2 s = scorer.score(&big);
    uint32_t mn = 0xffffffffu, mx = 0;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int j = j0 + 8 * r;
      const float x = r ? s.y : s.x;
      if ((lane & 3) == 0 && j < blocks) a.scores[row * a.max_blocks + j] = x;
      if (j >= a.n_first && j < c1) {
        const uint32_t key = key32(x);
        mn = min(mn, key);
        mx = max(mx, key);
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) big = MinMax<float>::mx(big, __shfl_xor_sync(kFull, big, o));
    mn = __reduce_min_sync(kFull, mn);
    mx = __reduce_max_sync(kFull, mx);
    if (lane == 0) a.stats[row * a.tiles + at] = TileStats{mn, mx, big, 0.f};
    if (!more) break;
    if (other) scorer.group(a, b, g);
  }
}

// The score of block j in 64 bits, as a key (in all lanes of the warp).  q:
// the group's rows in 64 bits, in shared memory.  kFinite: no infinity or NaN
// is among the row's values, so the product with zero need not be formed.
template <typename T, int D, int G, bool kFinite>
__device__ __forceinline__ uint64_t fine_key(const SelectArgs& a, const double (&q)[G][D], int b, int g, int j) {
  constexpr int kPer = D / 32;  // a lane's channels, adjacent
  const int lane = threadIdx.x & 31, d0 = lane * kPer;
  const int64_t tile = bounds_tile(a, a.block_tables[static_cast<int64_t>(b) * a.max_blocks + j], g);
  const T* src = static_cast<const T*>(a.bounds) + tile * 2 * D + d0;
  using C = Chunk<T, kPer>;
  C lows, highs;
  lows.raw = *reinterpret_cast<const typename C::Raw*>(src);
  highs.raw = *reinterpret_cast<const typename C::Raw*>(src + D);
  double s[G];
#pragma unroll
  for (int h = 0; h < G; ++h) s[h] = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const double lo = bound_value(lows.e[i]), hi = bound_value(highs.e[i]);
#pragma unroll
    for (int h = 0; h < G; ++h) {
      const double x = q[h][d0 + i];
      const bool down = __double2hiint(x) < 0;  // by the sign bit: a comparison would cost as much as a product
      if constexpr (kFinite) s[h] += x * (down ? lo : hi);
      else s[h] += (down ? x : 0.0) * lo + (down ? 0.0 : x) * hi;
    }
  }
  // sums over the lanes: while there are heads to share out, a lane keeps
  // half of them and passes the other half on
  int n = G;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    if (n > 1) {
      n >>= 1;
      const bool up = lane & o;
#pragma unroll
      for (int h = 0; h < G / 2; ++h)
        if (h < n) s[h] = (up ? s[h + n] : s[h]) + __shfl_xor_sync(kFull, up ? s[h] : s[h + n], o);
    } else {
      s[0] += __shfl_xor_sync(kFull, s[0], o);
    }
  }
  uint64_t best = key64(s[0]);
#pragma unroll
  for (int o = 16; o > 16 / G; o >>= 1) {
    const uint64_t y = __shfl_xor_sync(kFull, best, o);
    best = y > best ? y : best;
  }
  return best;
}

// Finds in hist[0 .. kBins) (counts per bin, larger keys in higher bins) the
// bin in which the need-th largest lies; *above: the count in higher bins.
// One count must reach `need`.
template <int kThreads, int kBins>
__device__ __forceinline__ int find_bin(const int* hist, int need, int* above, int* red, int* two) {
  constexpr int kPer = kBins / kThreads;
  const int top = kBins - 1 - static_cast<int>(threadIdx.x) * kPer;  // this thread's highest bin
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int h[kPer], mine = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) mine += h[i] = hist[top - i];
  int before = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, before, o);
    if (lane >= o) before += y;
  }
  if (lane == 31) red[warp] = before;
  __syncthreads();
  before += __reduce_add_sync(kFull, lane < warp ? red[lane] : 0) - mine;
  if (before < need && before + mine >= need) {
    int run = before, bin = top;
#pragma unroll
    for (int i = 0; i < kPer - 1; ++i)
      if (bin == top - i && run + h[i] < need) {
        run += h[i];
        --bin;
      }
    two[0] = bin;
    two[1] = run;
  }
  __syncthreads();
  *above = two[1];
  return two[0];
}

template <typename T, int D, int G, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 1024 ? 1 : 4) select_kernel(const SelectArgs a) {
  using Q = typename QueryOf<T>::type;
  constexpr int kWarps = kThreads / 32;
  extern __shared__ uint32_t bitmap[];  // one bit per block, then the scores of up to smem_scores blocks
  __shared__ int hist[kSelectBins];
  __shared__ uint64_t fine[kSelectFine];
  __shared__ int fine_at[kSelectFine];
  __shared__ int red[kWarps], two[2], count[2];
  __shared__ TileStats warp_stats[kWarps];
  __shared__ double q_fine[G][D];
  __shared__ float q_norm[G];
  // Behind score_kernel, which lets this grid be scheduled only once everything
  // before it is complete, q and the lengths may be read (from L2) while the
  // scores are still being computed.
  auto wait = [] {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  };
  if (!a.after_scores) wait();
  const int64_t row = blockIdx.x;
  const int b = static_cast<int>(row / a.num_kv_heads), g = static_cast<int>(row - static_cast<int64_t>(b) * a.num_kv_heads);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp < G) {  // q in 64 bits, and sum |q| of each head for the error bound
    float s = 0.f;
#pragma unroll
    for (int d = 0; d < D; d += 32) {
      const float x =
          widen1<Q>(__ldcg(static_cast<const Q*>(a.q) + (static_cast<int64_t>(b) * a.num_q_heads + g * G + warp) * D + d + lane));
      q_fine[warp][d + lane] = x;
      s += fabsf(x);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
    if (lane == 0) q_norm[warp] = s;
  }
  const int nblk = blocks_of(a, __ldcg(a.seq_lens + b), g == 0 && tid == 0);
  const int K = a.max_selected;
  int32_t* out = a.selected + row * K;
  if (nblk <= K) {  // every block
    if (a.after_scores) wait();
    for (int i = tid; i < K; i += kThreads) out[i] = i < nblk ? i : -1;
    return;
  }
  const int c0 = a.n_first, c1 = nblk - a.n_last;  // the candidates: more than are needed, since nblk > K
  const int need0 = K - a.n_first - a.n_last;
  const float* row_scores = a.scores + row * a.max_blocks;
  const int words = (nblk + 31) / 32;
  for (int i = tid; i < words; i += kThreads) {  // the first and the last blocks
    uint32_t m = 0;
    if (i * 32 < c0) m |= c0 - i * 32 >= 32 ? kFull : (1u << (c0 - i * 32)) - 1;
    if (i * 32 + 32 > c1) m |= c1 <= i * 32 ? kFull : kFull << (c1 - i * 32);
    if (i == words - 1 && (nblk & 31)) m &= (1u << (nblk & 31)) - 1;
    bitmap[i] = m;
  }
  if (a.after_scores) wait();

  if (need0 > 0) {
    const float* scores = row_scores;
    if (nblk <= a.smem_scores) {
      float* copy = reinterpret_cast<float*>(bitmap + (a.max_blocks + 31) / 32);
      for (int j = tid; j < nblk; j += kThreads) copy[j] = row_scores[j];
      scores = copy;
    }
    {
      uint32_t mn = 0xffffffffu, mx = 0;
      float big = 0.f;
      for (int t = tid; t < (nblk + 15) / 16; t += kThreads) {
        const TileStats st = a.stats[row * a.tiles + t];
        mn = min(mn, st.min_key);
        mx = max(mx, st.max_key);
        big = MinMax<float>::mx(big, st.big);
      }
      mn = __reduce_min_sync(kFull, mn);
      mx = __reduce_max_sync(kFull, mx);
#pragma unroll
      for (int o = 16; o; o >>= 1) big = MinMax<float>::mx(big, __shfl_xor_sync(kFull, big, o));
      if (lane == 0) warp_stats[warp] = TileStats{mn, mx, big, 0.f};
    }
    for (int i = tid; i < kSelectBins; i += kThreads) hist[i] = 0;
    if (tid < 2) count[tid] = 0;
    __syncthreads();
    const TileStats st = warp_stats[lane % kWarps];
    uint32_t base = __reduce_min_sync(kFull, st.min_key), last = __reduce_max_sync(kFull, st.max_key);
    float big = st.big, q1 = q_norm[lane % G];
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      big = MinMax<float>::mx(big, __shfl_xor_sync(kFull, big, o));
      q1 = MinMax<float>::mx(q1, __shfl_xor_sync(kFull, q1, o));
    }
    const float eps = q1 * big * kScoreError + kScoreTiny;
    const bool bounded = eps <= 1e30f;  // false for infinities and NaN: every candidate is scored in 64 bits

    // ---- narrow the keys' range to a bin that holds the need0-th largest ----
    float t_lo = -INFINITY, t_hi = INFINITY;  // the need0-th largest score lies in [t_lo, t_hi]
    if (bounded) {
      int need = need0;
      for (;;) {  // each round keeps less than 1 / 512 of the range
        int shift = 0;
        while (((last - base) >> shift) >= kSelectBins) ++shift;
        for (int j = c0 + tid; j < c1; j += kThreads) {
          const uint32_t k = key32(scores[j]);
          if (k >= base && k <= last) atomicAdd(&hist[(k - base) >> shift], 1);
        }
        __syncthreads();
        int above;
        const int bin = find_bin<kThreads, kSelectBins>(hist, need, &above, red, two);
        const int in_bin = hist[bin];
        need -= above;
        base += static_cast<uint32_t>(bin) << shift;
        const uint32_t width = (1u << shift) - 1;
        if (last - base > width) last = base + width;
        if (shift == 0 || in_bin <= 8) break;
        __syncthreads();
        for (int i = tid; i < kSelectBins; i += kThreads) hist[i] = 0;
        __syncthreads();
      }
      t_lo = unkey32(base);
      t_hi = unkey32(last);
    }

    // ---- blocks surely in, and those near the border ----
    // A 64-bit score is within eps of its 32-bit one.  Fewer than need0 blocks
    // score above t_hi, so the need0-th largest 64-bit score is at most
    // t_hi + eps, and likewise at least t_lo - eps.
    const float in_above = bounded ? t_hi + 2.f * eps : INFINITY;
    const float out_below = bounded ? t_lo - 2.f * eps : -INFINITY;
    for (int j0 = 0; j0 < words * 32; j0 += kThreads) {
      const int j = j0 + tid;
      bool in = false, near = false;
      if (j >= c0 && j < c1) {
        const float s = scores[j];
        in = bounded && s > in_above;
        near = !in && !(bounded && s < out_below);
      }
      const uint32_t m = __ballot_sync(kFull, in);
      if (lane == 0 && m) {
        bitmap[j >> 5] |= m;
        atomicAdd(&count[1], __popc(m));
      }
      if (near) {
        const int at = atomicAdd(&count[0], 1);
        if (at < kSelectFine) fine_at[at] = j;
      }
    }
    __syncthreads();
    const int n_near = count[0], need = need0 - count[1];  // of the near blocks

    if (n_near <= kSelectFine) {
      if (n_near > need) {
        for (int i = warp; i < n_near; i += kWarps) {
          const int j = fine_at[i];
          const uint64_t k =
              bounded ? fine_key<T, D, G, true>(a, q_fine, b, g, j) : fine_key<T, D, G, false>(a, q_fine, b, g, j);
          if (lane == 0) fine[i] = k;
        }
        __syncthreads();
      }
      for (int i = tid; i < n_near; i += kThreads) {
        const int j = fine_at[i];
        int rank_of = 0;
        if (n_near > need) {
          const uint64_t k = fine[i];
          for (int x = 0; x < n_near; ++x) rank_of += fine[x] > k || (fine[x] == k && fine_at[x] < j);
        }
        if (rank_of < need) atomicOr(&bitmap[j >> 5], 1u << (j & 31));
      }
    } else {
      // many blocks within the error of the border (equal keys, infinities):
      // 64-bit keys in the workspace and a radix selection over them
      uint64_t* keys = a.fine + row * a.max_blocks;
      for (int j = c0 + warp; j < c1; j += kWarps) {
        const float s = scores[j];
        if (bounded && (s > in_above || s < out_below)) continue;
        const uint64_t k = fine_key<T, D, G, false>(a, q_fine, b, g, j);
        if (lane == 0) keys[j] = k;
      }
      __syncthreads();
      uint64_t prefix = 0;
      int left = need;
      for (int shift = 56; shift >= 0; shift -= 8) {
        for (int i = tid; i < kSelectBins; i += kThreads) hist[i] = 0;  // 256 of them in use
        __syncthreads();
        for (int j = c0 + tid; j < c1; j += kThreads) {
          const float s = scores[j];
          if (bounded && (s > in_above || s < out_below)) continue;
          const uint64_t k = keys[j];
          if (shift == 56 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(k >> shift) & 255], 1);
        }
        __syncthreads();
        int above;
        const int bin = find_bin<kThreads, kSelectBins>(hist, left, &above, red, two);
        left -= above;
        prefix |= static_cast<uint64_t>(bin) << shift;
        __syncthreads();
      }
      // keys above `prefix`, and the first `left` equal to it
      int equal = 0;
      for (int j0 = 0; j0 < words * 32; j0 += kThreads) {
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
        const int of = lane < kWarps ? red[lane] : 0;
        const int before = equal + __popc(me & ((1u << lane) - 1)) + __reduce_add_sync(kFull, lane < warp ? of : 0);
        equal += __reduce_add_sync(kFull, of);
        const uint32_t m = __ballot_sync(kFull, in || (eq && before < left));
        if (lane == 0 && m) bitmap[j >> 5] |= m;
      }
    }
  }
  __syncthreads();

  // ---- the bitmap as an ascending list ----
  int done = 0;
  for (int w0 = 0; w0 < words; w0 += kThreads) {
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
    const int of = lane < kWarps ? red[lane] : 0;
    at += done - n + __reduce_add_sync(kFull, lane < warp ? of : 0);
    done += __reduce_add_sync(kFull, of);
    while (m) {
      if (at < K) out[at] = w * 32 + __ffs(m) - 1;
      ++at;
      m &= m - 1;
    }
  }
}

}  // namespace pkv
