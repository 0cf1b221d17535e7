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
// rotated one).  A token's R/2 angles are computed once by its CTA and shared
// by all its heads through shared memory; a thread then moves "units" of two
// 16-byte chunks that hold both halves of the pairs, so a rotation needs no
// exchange between threads and may run in place.
#pragma once

#include <cuda_fp8.h>

#include <type_traits>

#include "device_common.cuh"

namespace pkv {

constexpr int kRopeThreads = 128;
constexpr int kRopeMaxPairs = 512;  // channel pairs of the tokens of one CTA (shared memory: 8 bytes each)

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

// How a row is cut into units.  Half layout: unit u < half / kVec rotates
// chunk u with chunk u + half / kVec; the chunks from 2 half / kVec on pass
// through in twos.  Interleaved: pairs lie inside a chunk, and unit u takes
// chunks u and u + ceil(chunks / 2).  V rows likewise, unrotated.
struct UnitMap {
  int32_t chunks, rot, units;  // chunks of a row; units that pair up rotated halves; units of a row
};

template <int kVec, bool kInterleaved>
__device__ __forceinline__ UnitMap unit_map(int head_dim, int half) {
  UnitMap m;
  m.chunks = head_dim / kVec;
  m.rot = kInterleaved ? 0 : half / kVec;
  m.units = m.rot + (m.chunks - 2 * m.rot + 1) / 2;
  return m;
}

// kPool: 0 rotates q only; 1 also appends k and v to a pool of type T;
// 2 to an e4m3 pool.
template <typename T, typename TQ, int kVec, bool kInterleaved, int kPool>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs a) {
  __shared__ float2 cs[kRopeMaxPairs];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tok0 = blockIdx.x * a.tokens_per_cta;
  const int ntok = min(a.tokens_per_cta, a.n_tokens - tok0);
  const UnitMap rm = unit_map<kVec, kInterleaved>(a.head_dim, a.half);
  const int vunits = (rm.chunks + 1) / 2;
  const int q_units = a.num_q_heads * rm.units;
  const int k_units = kPool ? a.num_kv_heads * rm.units : 0;
  const int per_token = q_units + k_units + (kPool ? a.num_kv_heads * vunits : 0);

  for (int i = threadIdx.x; i < ntok * a.half; i += kRopeThreads) {
    const int t = i / a.half, p = i - t * a.half;
    const double turns = static_cast<double>(a.positions[tok0 + t]) * a.inv_freq[p] * 0.15915494309189533577;
    const float r = static_cast<float>(turns - rint(turns));  // in [-0.5, 0.5]
    float s, c;
    sincospif(2.0f * r, &s, &c);
    cs[i] = make_float2(c * a.factor, s * a.factor * a.sin_sign);
  }
  __syncthreads();

  for (int u0 = threadIdx.x; u0 < ntok * per_token; u0 += kRopeThreads) {
    const int t = u0 / per_token;
    int u = u0 - t * per_token;
    const int64_t tok = tok0 + t;
    // which row: 0 q, 1 k, 2 v
    int kind = 0;
    if (kPool && u >= q_units) {
      u -= q_units;
      kind = 1;
      if (u >= k_units) {
        u -= k_units;
        kind = 2;
      }
    }
    const int units = kind == 2 ? vunits : rm.units;
    const int h = u / units;
    u -= h * units;
    int c0, c1;
    bool rotate;
    if (kind == 2 || kInterleaved) {
      c0 = u;
      c1 = u + (rm.chunks + 1) / 2;
      rotate = kInterleaved && kind != 2;
    } else if (u < rm.rot) {
      c0 = u;
      c1 = u + rm.rot;
      rotate = true;
    } else {
      const int rest = rm.chunks - 2 * rm.rot;
      c0 = 2 * rm.rot + (u - rm.rot);
      c1 = c0 + (rest + 1) / 2;
      rotate = false;
    }
    const bool two = c1 < rm.chunks;
    int64_t dst = 0;  // of the row in its pool, elements
    if (kPool && kind) {
      const int32_t slot = a.slots[tok];
      if (slot < 0) continue;
      const int32_t blk = slot / a.block_size, off = slot - blk * a.block_size;
      if (blk >= a.num_blocks) {
        if (kind == 1 && h == 0 && u == 0) record_error(PKV_ERR_BAD_BLOCK);
        continue;
      }
      dst = ((static_cast<int64_t>(blk) * a.num_kv_heads + h) * a.block_size + off) * a.head_dim;
    }
    using C = Chunk<T, kVec>;
    const T* src = kind == 0 ? static_cast<const T*>(a.q) + tok * a.q_stride
                             : (kind == 1 ? static_cast<const T*>(a.k) + tok * a.k_stride
                                          : static_cast<const T*>(a.v) + tok * a.v_stride);
    src += h * a.head_dim;
    C x0, x1;
    x0.raw = *reinterpret_cast<const typename C::Raw*>(src + c0 * kVec);
    if (two) x1.raw = *reinterpret_cast<const typename C::Raw*>(src + c1 * kVec);
    else x1 = x0;

    float f0[kVec], f1[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      f0[i] = widen1<T>(x0.e[i]);
      f1[i] = widen1<T>(x1.e[i]);
    }
    if (rotate) {
      const float2* tc = cs + t * a.half;
      if constexpr (kInterleaved) {
#pragma unroll
        for (int i = 0; i < kVec; i += 2) {
          const int p0 = (c0 * kVec + i) >> 1, p1 = (c1 * kVec + i) >> 1;
          if (p0 < a.half) {
            const float2 w = tc[p0];
            const float xa = f0[i], xb = f0[i + 1];
            f0[i] = xa * w.x - xb * w.y;
            f0[i + 1] = xa * w.y + xb * w.x;
            x0.e[i] = narrow1<T>(f0[i]);
            x0.e[i + 1] = narrow1<T>(f0[i + 1]);
          }
          if (two && p1 < a.half) {
            const float2 w = tc[p1];
            const float xa = f1[i], xb = f1[i + 1];
            f1[i] = xa * w.x - xb * w.y;
            f1[i + 1] = xa * w.y + xb * w.x;
            x1.e[i] = narrow1<T>(f1[i]);
            x1.e[i + 1] = narrow1<T>(f1[i + 1]);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          const float2 w = tc[c0 * kVec + i];
          const float xa = f0[i], xb = f1[i];
          f0[i] = xa * w.x - xb * w.y;
          f1[i] = xa * w.y + xb * w.x;
          x0.e[i] = narrow1<T>(f0[i]);
          x1.e[i] = narrow1<T>(f1[i]);
        }
      }
    }

    if (kind == 0) {
      TQ* out = static_cast<TQ*>(a.q_out) + tok * a.out_stride + h * a.head_dim;
      if constexpr (std::is_same_v<T, TQ>) {  // channels that pass through keep their bits
        *reinterpret_cast<typename C::Raw*>(out + c0 * kVec) = x0.raw;
        if (two) *reinterpret_cast<typename C::Raw*>(out + c1 * kVec) = x1.raw;
      } else {
        using CQ = Chunk<TQ, kVec>;
        CQ y0, y1;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          y0.e[i] = narrow1<TQ>(f0[i]);
          y1.e[i] = narrow1<TQ>(f1[i]);
        }
        *reinterpret_cast<typename CQ::Raw*>(out + c0 * kVec) = y0.raw;
        if (two) *reinterpret_cast<typename CQ::Raw*>(out + c1 * kVec) = y1.raw;
      }
    } else if constexpr (kPool == 1) {
      T* out = static_cast<T*>(kind == 1 ? a.k_pool : a.v_pool) + dst;
      *reinterpret_cast<typename C::Raw*>(out + c0 * kVec) = x0.raw;
      if (two) *reinterpret_cast<typename C::Raw*>(out + c1 * kVec) = x1.raw;
    } else if constexpr (kPool == 2) {
      // the rotated value is rounded once, straight to its e4m3 code
      uint8_t* out = static_cast<uint8_t*>(kind == 1 ? a.k_pool : a.v_pool) + dst;
      const float inv = kind == 1 ? a.k_inv : a.v_inv;
      using C8 = Chunk<uint8_t, kVec>;
      C8 y0, y1;
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        y0.e[i] = __nv_cvt_float_to_fp8(f0[i] * inv, __NV_SATFINITE, __NV_E4M3);
        y1.e[i] = __nv_cvt_float_to_fp8(f1[i] * inv, __NV_SATFINITE, __NV_E4M3);
      }
      *reinterpret_cast<typename C8::Raw*>(out + c0 * kVec) = y0.raw;
      if (two) *reinterpret_cast<typename C8::Raw*>(out + c1 * kVec) = y1.raw;
    }
  }
}

}  // namespace pkv
