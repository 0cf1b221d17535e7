// Entry points of the rotary operators (included by pkv_device.cu).
#pragma once

namespace {

// A tensor of rows [n_tokens][heads][head_dim] whose tokens lie `stride`
// elements apart.
int check_rows(const char* fn, const char* what, const void* p, int64_t stride, int64_t heads, int32_t head_dim,
               int dtype) {
  if (!p) return fail(PKV_ERR_INVALID_ARG, "%s: %s is NULL", fn, what);
  if (!aligned16(p)) return fail(PKV_ERR_INVALID_ARG, "%s: %s must be 16-byte aligned", fn, what);
  if (stride < heads * head_dim)
    return fail(PKV_ERR_INVALID_ARG, "%s: the token stride of %s is less than a token", fn, what);
  if (stride * static_cast<int64_t>(elem_size(dtype)) % 16 != 0)
    return fail(PKV_ERR_INVALID_ARG, "%s: the token stride of %s must be a multiple of 16 bytes", fn, what);
  return PKV_OK;
}

int check_rotation(const char* fn, int32_t n_tokens, const int32_t* positions, const double* inv_freq,
                   int32_t head_dim, int32_t rot_dim, int32_t interleaved, float factor) {
  if (rot_dim <= 0 || rot_dim % 2 != 0 || rot_dim > head_dim)
    return fail(PKV_ERR_INVALID_ARG, "%s: rot_dim %d must be even, positive and at most head_dim %d", fn, rot_dim,
                head_dim);
  if (interleaved != 0 && interleaved != 1) return fail(PKV_ERR_INVALID_ARG, "%s: interleaved must be 0 or 1", fn);
  if (!std::isfinite(factor)) return fail(PKV_ERR_INVALID_ARG, "%s: factor is not finite", fn);
  if (n_tokens > 0 && (!positions || !inv_freq)) return fail(PKV_ERR_INVALID_ARG, "%s: NULL pointer", fn);
  if ((reinterpret_cast<uintptr_t>(inv_freq) & 7u) != 0)
    return fail(PKV_ERR_INVALID_ARG, "%s: inv_freq must be 8-byte aligned", fn);
  return PKV_OK;
}

template <typename T, typename TQ, int kPool>
int launch_rope(pkv::RopeArgs a, bool interleaved, const char* fn, cudaStream_t s) {
  constexpr int kVec = 16 / sizeof(T);
  // 16-byte chunks where they pair up; a half that is no multiple of a chunk
  // moves element by element: 8192 tokens of 32 bf16 heads of 128 take 24.8 us
  // with 128 rotated channels and 65 to 67 with 20, 24 or 124 (appended with 8 + 8
  // KV heads 39 and 125, to e4m3 pools 42 and 130).
  const bool vec = interleaved || a.half % kVec == 0;
  const int chunks = a.head_dim / (vec ? kVec : 1), units = (chunks + 1) / 2;
  const int rows = a.num_q_heads + (kPool ? 2 * a.num_kv_heads : 0);
  const int threads = units > pkv::kRopeThreads ? 2 * pkv::kRopeThreads : pkv::kRopeThreads;
  // tokens of a CTA: what fills its lines, and more where there are enough for
  // eight CTAs an SM all the same
  const int lines = threads / units;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  const int want = std::max(std::max(1, lines / rows), std::min(4, a.n_tokens / (8 * sm_count(dev))));
  a.tokens_per_cta = std::min(std::min(want, pkv::kRopeMaxTokens), std::max(1, pkv::kRopeMaxPairs / a.half));
  const dim3 grid(static_cast<unsigned>((a.n_tokens + a.tokens_per_cta - 1) / a.tokens_per_cta)),
      block(static_cast<unsigned>(threads));
  if (interleaved) e = launch_pdl(pkv::rope_kernel<T, TQ, kVec, true, kPool>, grid, block, 0, s, a);
  else if (vec) e = launch_pdl(pkv::rope_kernel<T, TQ, kVec, false, kPool>, grid, block, 0, s, a);
  else e = launch_pdl(pkv::rope_kernel<T, TQ, 1, false, kPool>, grid, block, 0, s, a);
  if (e != cudaSuccess) return cuda_fail(e, fn);
  return pkv::ok();
}

int rope_append(const char* fn, const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                int64_t v_stride, const int32_t* positions, const double* inv_freq, const int32_t* slot_mapping,
                int32_t n_tokens, void* q_out, void* k_pool, void* v_pool, int32_t num_blocks, int32_t num_q_heads,
                int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int32_t rot_dim, int32_t interleaved,
                float factor, int32_t src_dtype, bool fp8, float k_scale, float v_scale, void* stream) {
  int rc = check_common(num_kv_heads, head_dim, block_size, src_dtype, fn);
  if (rc) return rc;
  if (n_tokens < 0 || num_blocks <= 0 || num_q_heads < 0 || num_q_heads > 65536 || num_kv_heads > 65536)
    return fail(PKV_ERR_INVALID_ARG, "%s: bad sizes", fn);
  rc = check_rotation(fn, n_tokens, positions, inv_freq, head_dim, rot_dim, interleaved, factor);
  if (rc) return rc;
  if (fp8 && (!(k_scale > 0.f) || !(v_scale > 0.f) || !std::isfinite(k_scale) || !std::isfinite(v_scale)))
    return fail(PKV_ERR_INVALID_ARG, "%s: scales must be positive and finite", fn);
  if (n_tokens == 0) return pkv::ok();
  if (num_q_heads > 0) {
    rc = check_rows(fn, "q", q, q_stride, num_q_heads, head_dim, src_dtype);
    if (rc) return rc;
    if (!q_out || !aligned16(q_out)) return fail(PKV_ERR_INVALID_ARG, "%s: q_out is NULL or not 16-byte aligned", fn);
  }
  rc = check_rows(fn, "k", k, k_stride, num_kv_heads, head_dim, src_dtype);
  if (rc) return rc;
  rc = check_rows(fn, "v", v, v_stride, num_kv_heads, head_dim, src_dtype);
  if (rc) return rc;
  if (!slot_mapping || !k_pool || !v_pool) return fail(PKV_ERR_INVALID_ARG, "%s: NULL pointer", fn);
  if (!aligned16(k_pool) || !aligned16(v_pool))
    return fail(PKV_ERR_INVALID_ARG, "%s: pools must be 16-byte aligned", fn);
  pkv::RopeArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.out_stride = static_cast<int64_t>(num_q_heads) * head_dim;
  a.positions = positions;
  a.inv_freq = inv_freq;
  a.slots = slot_mapping;
  a.q_out = q_out;
  a.k_pool = k_pool;
  a.v_pool = v_pool;
  a.n_tokens = n_tokens;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = num_kv_heads;
  a.head_dim = head_dim;
  a.half = rot_dim / 2;
  a.num_blocks = num_blocks;
  a.block_size = block_size;
  a.factor = factor;
  a.sin_sign = 1.0f;
  a.k_inv = fp8 ? static_cast<float>(1.0 / static_cast<double>(k_scale)) : 1.0f;
  a.v_inv = fp8 ? static_cast<float>(1.0 / static_cast<double>(v_scale)) : 1.0f;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool il = interleaved != 0;
  if (fp8) {
    switch (src_dtype) {
      case PKV_F32: return launch_rope<float, __half, 2>(a, il, fn, s);
      case PKV_BF16: return launch_rope<__nv_bfloat16, __half, 2>(a, il, fn, s);
      default: return launch_rope<__half, __half, 2>(a, il, fn, s);
    }
  }
  switch (src_dtype) {
    case PKV_F32: return launch_rope<float, float, 1>(a, il, fn, s);
    case PKV_BF16: return launch_rope<__nv_bfloat16, __nv_bfloat16, 1>(a, il, fn, s);
    default: return launch_rope<__half, __half, 1>(a, il, fn, s);
  }
}

}  // namespace

extern "C" int pkv_rope(const void* x, int64_t x_stride, const int32_t* positions, const double* inv_freq,
                        int32_t n_tokens, int32_t num_heads, int32_t head_dim, int32_t rot_dim, int32_t interleaved,
                        float factor, int32_t transpose, int32_t dtype, void* out, int64_t out_stride, void* stream) {
  const char* fn = "pkv_rope";
  NvtxRange nvtx_range(fn);
  if (dtype != PKV_F32 && dtype != PKV_BF16 && dtype != PKV_F16)
    return fail(PKV_ERR_UNSUPPORTED, "%s: dtype %d not supported", fn, dtype);
  if (head_dim <= 0 || head_dim % 8 != 0 || head_dim > 512)
    return fail(PKV_ERR_UNSUPPORTED, "%s: head_dim %d not supported (a multiple of 8, at most 512)", fn, head_dim);
  if (n_tokens < 0 || num_heads <= 0 || num_heads > 65536) return fail(PKV_ERR_INVALID_ARG, "%s: bad sizes", fn);
  if (transpose != 0 && transpose != 1) return fail(PKV_ERR_INVALID_ARG, "%s: transpose must be 0 or 1", fn);
  int rc = check_rotation(fn, n_tokens, positions, inv_freq, head_dim, rot_dim, interleaved, factor);
  if (rc) return rc;
  if (n_tokens == 0) return pkv::ok();
  rc = check_rows(fn, "x", x, x_stride, num_heads, head_dim, dtype);
  if (rc) return rc;
  rc = check_rows(fn, "out", out, out_stride, num_heads, head_dim, dtype);
  if (rc) return rc;
  if (x == out && x_stride != out_stride)
    return fail(PKV_ERR_INVALID_ARG, "%s: in place, x and out need the same token stride", fn);
  pkv::RopeArgs a{};
  a.q = x;
  a.q_stride = x_stride;
  a.out_stride = out_stride;
  a.positions = positions;
  a.inv_freq = inv_freq;
  a.q_out = out;
  a.n_tokens = n_tokens;
  a.num_q_heads = num_heads;
  a.head_dim = head_dim;
  a.half = rot_dim / 2;
  a.factor = factor;
  a.sin_sign = transpose ? -1.0f : 1.0f;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool il = interleaved != 0;
  switch (dtype) {
    case PKV_F32: return launch_rope<float, float, 0>(a, il, fn, s);
    case PKV_BF16: return launch_rope<__nv_bfloat16, __nv_bfloat16, 0>(a, il, fn, s);
    default: return launch_rope<__half, __half, 0>(a, il, fn, s);
  }
}

extern "C" int pkv_rope_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                               int64_t v_stride, const int32_t* positions, const double* inv_freq,
                               const int32_t* slot_mapping, int32_t n_tokens, void* q_out, void* k_pool, void* v_pool,
                               int32_t num_blocks, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                               int32_t block_size, int32_t rot_dim, int32_t interleaved, float factor, int32_t dtype,
                               void* stream) {
  const char* fn = "pkv_rope_append";
  NvtxRange nvtx_range(fn);
  return rope_append(fn, q, q_stride, k, k_stride, v, v_stride, positions, inv_freq, slot_mapping, n_tokens, q_out,
                     k_pool, v_pool, num_blocks, num_q_heads, num_kv_heads, head_dim, block_size, rot_dim, interleaved,
                     factor, dtype, false, 1.f, 1.f, stream);
}

extern "C" int pkv_rope_append_fp8(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                   int64_t v_stride, int32_t src_dtype, const int32_t* positions,
                                   const double* inv_freq, const int32_t* slot_mapping, int32_t n_tokens, void* q_out,
                                   void* k_pool, void* v_pool, int32_t num_blocks, int32_t num_q_heads,
                                   int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int32_t rot_dim,
                                   int32_t interleaved, float factor, float k_scale, float v_scale, void* stream) {
  const char* fn = "pkv_rope_append_fp8";
  NvtxRange nvtx_range(fn);
  return rope_append(fn, q, q_stride, k, k_stride, v, v_stride, positions, inv_freq, slot_mapping, n_tokens, q_out,
                     k_pool, v_pool, num_blocks, num_q_heads, num_kv_heads, head_dim, block_size, rot_dim, interleaved,
                     factor, src_dtype, true, k_scale, v_scale, stream);
}
