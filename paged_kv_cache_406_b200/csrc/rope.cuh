// Rotary positions, alone or on the way into the paged pool.
//
// For channel pair i of a head (half layout: channels i and i + R/2;
// interleaved: 2i and 2i + 1; R rotated channels, the others pass through)
// and a token at position p,
//     angle = p * inv_freq[i],  c = factor * cos(angle),  s = factor * sin(angle)
//     y_a = x_a c - x_b s,      y_b = x_a s + x_b c
// The transposed map (s negated) takes the gradient of y to that of x.
//
// The angle is formed and reduced to a fraction of a turn in 64 bits, so far
// positions keep their phase (p = 2^20 in 32 bits would be off by up to 0.06
// rad); the sine and cosine of the reduced angle, the products and the sums
// are 32-bit, and each output is rounded once.
//
// What bounds it: bytes (each element is read and written once, 3 flops per
// rotated one).  A CTA takes a few tokens: it issues the loads of the first
// rows, computes the tokens' angles once for all heads under them, and shares
// them through shared memory.  A thread keeps to one unit of every row it
// moves, two 16-byte chunks that hold both halves of its pairs: a token's sines
// and cosines stay in its registers, a rotation needs no exchange between
// threads and may run in place.  A row in flight per thread and many threads
// did better than two to four rows of fewer: 8192 tokens of 32 + 8 + 8 heads in
// 39.5 us (5.1 TB/s) against 44 to 48, four tokens a CTA against 41.5 for one.
#pragma once

#include <cuda_fp8.h>

#include <type_traits>

#include "device_common.cuh"

namespace pkv {

constexpr int kRopeThreads = 128;   // 256 where a row has more than 128 units
constexpr int kRopeMaxPairs = 512;  // channel pairs of the tokens of one CTA (shared memory: 8 bytes each)
constexpr int kRopeMaxTokens = 32;

struct RopeArgs {
  const void* q;
  const void* k;  // append only
  const void* v;
  int64_t q_stride, k_stride, v_stride, out_stride;  // elements between tokens
  const int32_t* positions;
  const double* inv_freq;
  const int32_t* slots;
  void* q_out;
  void* k_pool;
  void* v_pool;
  int32_t n_tokens, num_q_heads, num_kv_heads, head_dim, half;  // half = rotated channels / 2
  int32_t num_blocks, block_size;
  int32_t tokens_per_cta;
  float factor;     // > 0; the sine's sign is in sin_sign
  float sin_sign;   // -1: transposed
  float k_inv, v_inv;  // e4m3 only: 1 / scale
};

template <int kBytes>
struct RawOf;
template <>
struct RawOf<16> { using type = uint4; };
template <>
struct RawOf<8> { using type = uint2; };
template <>
struct RawOf<4> { using type = uint32_t; };
template <>
struct RawOf<2> { using type = uint16_t; };
template <>
struct RawOf<1> { using type = uint8_t; };

// kVec elements of T as one load or store.
template <typename T, int kVec>
struct Chunk {
  using Raw = typename RawOf<sizeof(T) * kVec>::type;
  union {
    Raw raw;
    T e[kVec];
  };
  __device__ __forceinline__ Chunk() {}
};

template <typename T>
__device__ __forceinline__ float widen1(T x) {
  if constexpr (std::is_same_v<T, float>) return x;
  else if constexpr (std::is_same_v<T, __half>) return __half2float(x);
  else return __bfloat162float(x);
}

template <typename T>
__device__ __forceinline__ T narrow1(float x) {
  if constexpr (std::is_same_v<T, float>) return x;
  else if constexpr (std::is_same_v<T, __half>) return __float2half_rn(x);
  else return __float2bfloat16_rn(x);
}

// kVec floats as codes of T, or raw e4m3 codes.
template <typename T, int kVec>
__device__ __forceinline__ Chunk<T, kVec> narrow_chunk(const float (&f)[kVec]) {
  Chunk<T, kVec> c;
#pragma unroll
  for (int i = 0; i < kVec; ++i) c.e[i] = narrow1<T>(f[i]);
  return c;
}
template <int kVec>
__device__ __forceinline__ Chunk<uint8_t, kVec> e4m3_chunk(const float (&f)[kVec], float scale) {
  Chunk<uint8_t, kVec> c;
  if constexpr (kVec == 1) {
    c.e[0] = __nv_cvt_float_to_fp8(f[0] * scale, __NV_SATFINITE, __NV_E4M3);
  } else {
#pragma unroll
    for (int i = 0; i < kVec; i += 2) {
      const __nv_fp8x2_storage_t y = __nv_cvt_float2_to_fp8x2(make_float2(f[i] * scale, f[i + 1] * scale), __NV_SATFINITE, __NV_E4M3);
      c.e[i] = static_cast<uint8_t>(y);
      c.e[i + 1] = static_cast<uint8_t>(y >> 8);
    }
  }
  return c;
}

// kPool: 0 rotates q only; 1 also appends k and v to a pool of type T; 2 to an
// e4m3 pool.  A row is cut into units of two kVec-element chunks: in the half
// layout unit x < half / kVec holds chunk x and its partner x + half / kVec, the
// others two chunks that pass through; interleaved, pairs lie inside a chunk
// and the two are any.  V rows are cut the same way and pass through.
template <typename T, typename TQ, int kVec, bool kInterleaved, int kPool>
__global__ void __launch_bounds__(256) rope_kernel(const RopeArgs a) {
  using C = Chunk<T, kVec>;
  __shared__ float2 cs[kRopeMaxPairs];
  __shared__ int64_t place[kPool ? kRopeMaxTokens : 1];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int chunks = a.head_dim / kVec, units = (chunks + 1) / 2;
  const int rot = kInterleaved ? 0 : a.half / kVec;  // units that rotate (half layout)
  const int rows = a.num_q_heads + (kPool ? 2 * a.num_kv_heads : 0);
  const int lines = blockDim.x / units;              // rows the CTA moves at a time
  const int line = threadIdx.x / units, x = threadIdx.x - line * units;
  const int tok0 = blockIdx.x * a.tokens_per_cta;
  // this thread's rows: line, line + lines, ... of the tokens' rows in order;
  // none for the threads left over
  const int ntok = line < lines ? min(a.tokens_per_cta, a.n_tokens - tok0) : 0;
  const int dt = lines / rows, dr = lines - dt * rows;
  int t = line / rows, row = line - t * rows;

  int c0, c1;
  if (kInterleaved || x >= rot) {
    c0 = 2 * rot + (x - rot);
    c1 = c0 + (chunks - 2 * rot + 1) / 2;
  } else {
    c0 = x;
    c1 = x + rot;
  }
  const bool two = c1 < chunks;
  const int e0 = c0 * kVec, e1 = two ? c1 * kVec : c0 * kVec;

  auto source = [&](int t, int r) {
    const int64_t tok = tok0 + t;
    if (!kPool || r < a.num_q_heads) return static_cast<const T*>(a.q) + tok * a.q_stride + r * a.head_dim;
    r -= a.num_q_heads;
    if (r < a.num_kv_heads) return static_cast<const T*>(a.k) + tok * a.k_stride + r * a.head_dim;
    return static_cast<const T*>(a.v) + tok * a.v_stride + (r - a.num_kv_heads) * a.head_dim;
  };
  C x0, x1;
  auto load = [&] {
    if (t < ntok) {
      const T* src = source(t, row);
      x0.raw = *reinterpret_cast<const typename C::Raw*>(src + e0);
      x1.raw = *reinterpret_cast<const typename C::Raw*>(src + e1);
    }
  };
  load();

  const int held = min(a.tokens_per_cta, a.n_tokens - tok0);
  for (int i = threadIdx.x; i < held * a.half; i += blockDim.x) {
    const int ti = i / a.half, p = i - ti * a.half;
    const double turns = static_cast<double>(a.positions[tok0 + ti]) * a.inv_freq[p] * 0.15915494309189533577;
    const float r = static_cast<float>(turns - rint(turns));  // in [-0.5, 0.5]
    float s, c;
    sincospif(2.0f * r, &s, &c);
    cs[i] = make_float2(c * a.factor, s * a.factor * a.sin_sign);
  }
  if constexpr (kPool > 0) {  // head 0's row of each token in the pools, elements; -1: none
    for (int i = threadIdx.x; i < held; i += blockDim.x) {
      const int32_t slot = a.slots[tok0 + i];
      const int32_t blk = slot / a.block_size, off = slot - blk * a.block_size;
      const bool in = slot >= 0 && blk < a.num_blocks;
      if (slot >= 0 && !in) record_error(PKV_ERR_BAD_BLOCK);
      place[i] = in ? (static_cast<int64_t>(blk) * a.num_kv_heads * a.block_size + off) * a.head_dim : -1;
    }
  }
  __syncthreads();

  float2 w[kVec];                // of the unit's pairs
  const bool turn0 = kInterleaved ? e0 / 2 < a.half : x < rot;  // whether its chunks hold rotated channels
  const bool turn1 = kInterleaved ? two && e1 / 2 < a.half : turn0;
  int at = -1;                   // the token that w is of
  while (t < ntok) {
    const int kind = !kPool || row < a.num_q_heads ? 0 : (row < a.num_q_heads + a.num_kv_heads ? 1 : 2);
    const int64_t dst = kPool && kind ? place[t] : 0;
    if (at != t) {
      at = t;
      const float2* tc = cs + t * a.half;
      if constexpr (kInterleaved) {  // a chunk may be rotated in part
#pragma unroll
        for (int i = 0; i < kVec / 2; ++i) {
          if (turn0 && e0 / 2 + i < a.half) w[i] = tc[e0 / 2 + i];
          if (turn1 && e1 / 2 + i < a.half) w[kVec / 2 + i] = tc[e1 / 2 + i];
        }
      } else if (turn0) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) w[i] = tc[e0 + i];
      }
    }
    float f0[kVec], f1[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      f0[i] = widen1<T>(x0.e[i]);
      f1[i] = widen1<T>(x1.e[i]);
    }
    if (kind != 2) {
      if constexpr (kInterleaved) {
#pragma unroll
        for (int i = 0; i < kVec / 2; ++i) {
          if (turn0 && e0 / 2 + i < a.half) {
            const float xa = f0[2 * i], xb = f0[2 * i + 1];
            f0[2 * i] = xa * w[i].x - xb * w[i].y;
            f0[2 * i + 1] = xa * w[i].y + xb * w[i].x;
            x0.e[2 * i] = narrow1<T>(f0[2 * i]);
            x0.e[2 * i + 1] = narrow1<T>(f0[2 * i + 1]);
          }
          if (turn1 && e1 / 2 + i < a.half) {
            const float2 v = w[kVec / 2 + i];
            const float xa = f1[2 * i], xb = f1[2 * i + 1];
            f1[2 * i] = xa * v.x - xb * v.y;
            f1[2 * i + 1] = xa * v.y + xb * v.x;
            x1.e[2 * i] = narrow1<T>(f1[2 * i]);
            x1.e[2 * i + 1] = narrow1<T>(f1[2 * i + 1]);
          }
        }
      } else if (turn0) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          const float xa = f0[i], xb = f1[i];
          f0[i] = xa * w[i].x - xb * w[i].y;
          f1[i] = xa * w[i].y + xb * w[i].x;
        }
        x0 = narrow_chunk<T, kVec>(f0);
        x1 = narrow_chunk<T, kVec>(f1);
      }
    }
    if (dst < 0) {
      // a padding token's K and V go nowhere
    } else if (kind == 0) {
      TQ* out = static_cast<TQ*>(a.q_out) + (tok0 + static_cast<int64_t>(t)) * a.out_stride + row * a.head_dim;
      if constexpr (std::is_same_v<T, TQ>) {  // channels that pass through keep their bits
        *reinterpret_cast<typename C::Raw*>(out + e0) = x0.raw;
        if (two) *reinterpret_cast<typename C::Raw*>(out + e1) = x1.raw;
      } else {
        using CQ = Chunk<TQ, kVec>;
        *reinterpret_cast<typename CQ::Raw*>(out + e0) = narrow_chunk<TQ, kVec>(f0).raw;
        if (two) *reinterpret_cast<typename CQ::Raw*>(out + e1) = narrow_chunk<TQ, kVec>(f1).raw;
      }
    } else if constexpr (kPool > 0) {
      const int h = row - a.num_q_heads - (kind == 2 ? a.num_kv_heads : 0);
      const int64_t to = dst + static_cast<int64_t>(h) * a.block_size * a.head_dim;
      if constexpr (kPool == 1) {
        T* out = static_cast<T*>(kind == 1 ? a.k_pool : a.v_pool) + to;
        *reinterpret_cast<typename C::Raw*>(out + e0) = x0.raw;
        if (two) *reinterpret_cast<typename C::Raw*>(out + e1) = x1.raw;
      } else {  // the rotated value is rounded once, straight to its e4m3 code
        using C8 = Chunk<uint8_t, kVec>;
        uint8_t* out = static_cast<uint8_t*>(kind == 1 ? a.k_pool : a.v_pool) + to;
        const float inv = kind == 1 ? a.k_inv : a.v_inv;
        *reinterpret_cast<typename C8::Raw*>(out + e0) = e4m3_chunk<kVec>(f0, inv).raw;
        if (two) *reinterpret_cast<typename C8::Raw*>(out + e1) = e4m3_chunk<kVec>(f1, inv).raw;
      }
    }
    t += dt;
    row += dr;
    if (row >= rows) {
      row -= rows;
      ++t;
    }
    load();
  }
}

}  // namespace pkv
