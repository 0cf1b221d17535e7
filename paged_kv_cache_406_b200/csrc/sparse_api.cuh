// Entry points of block bounds, block selection and block-sparse decode
// (included by pkv_device.cu).
#pragma once

namespace {

constexpr int64_t kMaxSelectBlocks = int64_t(1) << 20;  // blocks of a sequence: a bit each in shared memory

// Sizes shared by the block-sparse calls; `pool_dtype` may be e4m3.
int check_sparse(const char* fn, int32_t num_seqs, int32_t num_kv_heads, int32_t head_dim, int32_t num_blocks,
                 int32_t max_blocks, int32_t block_size, int32_t pool_dtype) {
  const bool fp8 = pool_dtype == PKV_FP8_E4M3;
  int rc = check_common(num_kv_heads, head_dim, block_size, fp8 ? PKV_F16 : pool_dtype, fn);
  if (rc) return rc;
  if (fp8 && head_dim != 128) return fail(PKV_ERR_UNSUPPORTED, "%s: e4m3 pools need head_dim 128", fn);
  if (num_seqs < 0 || num_blocks <= 0 || max_blocks < 0) return fail(PKV_ERR_INVALID_ARG, "%s: bad sizes", fn);
  if (int64_t(max_blocks) * block_size > (int64_t(1) << 30) || max_blocks > kMaxSelectBlocks)
    return fail(PKV_ERR_INVALID_ARG, "%s: max_blocks_per_seq too large", fn);
  if (int64_t(num_seqs) * num_kv_heads > (int64_t(1) << 24))
    return fail(PKV_ERR_INVALID_ARG, "%s: num_seqs * num_kv_heads too large", fn);
  return PKV_OK;
}

int check_group(const char* fn, int32_t num_q_heads, int32_t num_kv_heads, bool f32) {
  if (num_q_heads <= 0 || num_q_heads % num_kv_heads != 0)
    return fail(PKV_ERR_INVALID_ARG, "%s: num_q_heads %d not a multiple of num_kv_heads %d", fn, num_q_heads,
                num_kv_heads);
  const int32_t group = num_q_heads / num_kv_heads;
  if (group != 1 && group != 2 && group != 4 && group != 8)
    return fail(PKV_ERR_UNSUPPORTED, "%s: group size %d not supported (1, 2, 4 or 8)", fn, group);
  if (group == 8 && f32) return fail(PKV_ERR_UNSUPPORTED, "%s: group size 8 needs 16-bit or e4m3 K/V", fn);
  return PKV_OK;
}

template <typename T, int D>
cudaError_t launch_bounds(const pkv::BoundsArgs& a, cudaStream_t s) {
  const int64_t warps = int64_t(a.num_seqs) * a.window * a.num_kv_heads;
  return launch_pdl(pkv::block_bounds_kernel<T, D>, dim3(static_cast<unsigned>((warps + 7) / 8)), dim3(256), 0, s, a);
}

struct SelectLayout {
  size_t stats, fine, total;  // byte offsets; the scores lie at 0
};

SelectLayout select_layout(int64_t rows, int64_t max_blocks) {
  SelectLayout w;
  w.stats = round256(static_cast<size_t>(rows * max_blocks) * sizeof(float));
  w.fine = w.stats + round256(static_cast<size_t>(rows * ((max_blocks + 15) / 16)) * sizeof(pkv::TileStats));
  w.total = w.fine + round256(static_cast<size_t>(rows * max_blocks) * sizeof(uint64_t));
  return w;
}

// Scores that a selecting CTA copies to shared memory: what leaves room for
// two CTAs on an SM.
constexpr int32_t kSelectSmemScores = 16384;

template <typename T, int D, int G>
int launch_select(pkv::SelectArgs a, const char* fn, cudaStream_t s) {
  const int64_t rows = int64_t(a.num_seqs) * a.num_kv_heads;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  const bool wide = rows <= sm_count(dev) && a.max_blocks > 2048;
  auto kern = wide ? pkv::select_kernel<T, D, G, 1024> : pkv::select_kernel<T, D, G, 256>;
  static std::atomic<bool> opted[kMaxDevices];
  if (dev >= kMaxDevices || !opted[dev].load(std::memory_order_relaxed)) {
    for (auto k : {pkv::select_kernel<T, D, G, 256>, pkv::select_kernel<T, D, G, 1024>}) {
      e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kMaxSelectBlocks / 8));
      if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(select)");
    }
    if (dev < kMaxDevices) opted[dev].store(true, std::memory_order_relaxed);
  }
  if (a.max_blocks > a.max_selected && a.max_selected > a.n_first + a.n_last) {  // else no score decides
    const int64_t ctas = (rows * a.tiles + pkv::kScoreWarps - 1) / pkv::kScoreWarps;  // a tile a warp
    e = launch_pdl(pkv::score_kernel<T, D, G>, dim3(static_cast<unsigned>(std::min<int64_t>(ctas, 2 * sm_count(dev)))),
                   dim3(pkv::kScoreThreads), 0, s, a);
    if (e != cudaSuccess) return cuda_fail(e, fn);
    a.after_scores = 1;
  }
  a.smem_scores = a.max_blocks <= kSelectSmemScores ? a.max_blocks : 0;
  const size_t smem = static_cast<size_t>((a.max_blocks + 31) / 32 + a.smem_scores) * 4;
  e = launch_pdl(kern, dim3(static_cast<unsigned>(rows)), dim3(wide ? 1024 : 256), smem, s, a);
  if (e != cudaSuccess) return cuda_fail(e, fn);
  return pkv::ok();
}

template <typename T, int D>
int launch_select_group(const pkv::SelectArgs& a, const char* fn, cudaStream_t s) {
  switch (a.num_q_heads / a.num_kv_heads) {
    case 1: return launch_select<T, D, 1>(a, fn, s);
    case 2: return launch_select<T, D, 2>(a, fn, s);
    case 4: return launch_select<T, D, 4>(a, fn, s);
    default: return launch_select<T, D, 8>(a, fn, s);
  }
}

struct SparseLayout {
  size_t lens, decode, total;  // byte offsets; the tables lie at 0
};

SparseLayout sparse_layout(int64_t rows, int32_t group, int32_t head_dim, int32_t max_selected, int32_t block_size,
                           int32_t pt) {
  SparseLayout w;
  w.lens = round256(static_cast<size_t>(rows) * max_selected * sizeof(int32_t));
  w.decode = w.lens + round256(static_cast<size_t>(rows) * sizeof(int32_t));
  w.total = w.decode + ws_layout(rows, group, 1, head_dim, int64_t(max_selected) * block_size, pt).total;
  return w;
}

template <typename T, int D, int G, int kWarps>
int launch_sparse(const pkv::SparseDecodeArgs& a, int ctas, int dev, const CUtensorMap& mk, const CUtensorMap& mv,
                  const char* fn, cudaStream_t s) {
  auto kern = pkv::sparse_decode_kernel<T, D, G, kWarps>;
  constexpr int kSmem = pkv::SparseSmem<T, D, G, kWarps>::kBytes;
  static std::atomic<bool> opted[kMaxDevices];
  cudaError_t e;
  if (dev >= kMaxDevices || !opted[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(sparse)");
    e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(carveout)");
    if (dev < kMaxDevices) opted[dev].store(true, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(int64_t(a.s.num_seqs) * a.s.num_kv_heads * ctas));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(ctas);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, kern, a, mk, mv);
  if (e != cudaSuccess) return cuda_fail(e, fn);
  return pkv::ok();
}

template <typename T, int D, int G>
int launch_sparse_shape(const pkv::SparseDecodeArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, const char* fn,
                        cudaStream_t s) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  const int64_t rows = int64_t(a.s.num_seqs) * a.s.num_kv_heads, sms = sm_count(dev);
  const int64_t chunks = (int64_t(a.s.max_selected) * a.s.block_size + 15) / 16;
  // CTAs of a row: as many as leave each warp a chunk and are resident at
  // once.  Eight-warp CTAs fill an SM, and clusters of eight do not pack the
  // SMs of a GPU partition: 16 rows of 256 blocks took 20 us in 16 clusters of
  // eight and 13.3 in clusters of four, 8 rows of 64 blocks 7.0 in clusters of
  // eight and 7.1 of four; 32 rows 8.6 in clusters of four and 9.2 of two.
  auto spread = [&](int warps, int64_t slots) {
    int ctas = 1;
    while (ctas < pkv::kSparseCluster && rows * ctas * 2 <= (ctas * 2 == 8 ? slots / 2 : slots) && chunks >= 2 * ctas * warps)
      ctas *= 2;
    return ctas;
  };
  if (rows <= sms) return launch_sparse<T, D, G, pkv::kSparseManyWarps>(a, spread(pkv::kSparseManyWarps, sms), dev, mk, mv, fn, s);
  return launch_sparse<T, D, G, pkv::kSparseFewWarps>(a, spread(pkv::kSparseFewWarps, 4 * sms), dev, mk, mv, fn, s);
}

template <typename T, int D>
int launch_sparse_group(const pkv::SparseDecodeArgs& a, const void* k_pool, const void* v_pool, int dtype, int32_t group,
                        const char* fn, cudaStream_t s) {
  const int64_t rows = int64_t(a.s.num_blocks) * a.s.num_kv_heads * a.s.block_size;
  const int box_rows = a.s.block_size < 16 ? a.s.block_size : 16;
  CUtensorMap mk, mv;
  int rc = pool_map(&mk, k_pool, dtype, rows, D, box_rows);
  if (rc) return rc;
  rc = pool_map(&mv, v_pool, dtype, rows, D, box_rows);
  if (rc) return rc;
  switch (group) {
    case 1: return launch_sparse_shape<T, D, 1>(a, mk, mv, fn, s);
    case 2: return launch_sparse_shape<T, D, 2>(a, mk, mv, fn, s);
    case 4: return launch_sparse_shape<T, D, 4>(a, mk, mv, fn, s);
    default: return launch_sparse_shape<T, D, 8>(a, mk, mv, fn, s);
  }
}

// The cluster kernel keeps a row's list in shared memory; 32-bit pools and
// longer lists run the dense kernels on the selection as a batch of its own.
bool sparse_by_cluster(int32_t dtype, int32_t max_selected) {
  return dtype != PKV_F32 && max_selected <= pkv::kSparseList;
}

int sparse_decode(const char* fn, const void* q, const void* k_pool, const void* v_pool, const int32_t* block_tables,
                  const int32_t* seq_lens, const int32_t* selected, int32_t max_selected, int32_t num_seqs,
                  int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t num_blocks, int32_t max_blocks,
                  int32_t block_size, float scale, int32_t dtype, float k_scale, float v_scale, void* workspace,
                  size_t workspace_bytes, float* out, void* stream) {
  int rc = check_sparse(fn, num_seqs, num_kv_heads, head_dim, num_blocks, max_blocks, block_size, dtype);
  if (rc) return rc;
  rc = check_group(fn, num_q_heads, num_kv_heads, dtype == PKV_F32);
  if (rc) return rc;
  if (max_selected <= 0 || int64_t(max_selected) * block_size > (int64_t(1) << 30))
    return fail(PKV_ERR_INVALID_ARG, "%s: max_selected %d", fn, max_selected);
  if (!std::isfinite(scale)) return fail(PKV_ERR_INVALID_ARG, "%s: scale is not finite", fn);
  if (!(k_scale > 0.f) || !(v_scale > 0.f) || !std::isfinite(k_scale) || !std::isfinite(v_scale))
    return fail(PKV_ERR_INVALID_ARG, "%s: k_scale and v_scale must be positive and finite", fn);
  if (int64_t(num_blocks) * num_kv_heads * block_size > INT32_MAX)
    return fail(PKV_ERR_INVALID_ARG, "%s: pool has more than 2^31 token rows", fn);
  if (num_seqs == 0) return pkv::ok();
  if (!q || !k_pool || !v_pool || !block_tables || !seq_lens || !selected || !out)
    return fail(PKV_ERR_INVALID_ARG, "%s: NULL pointer", fn);
  if (!aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(out))
    return fail(PKV_ERR_INVALID_ARG, "%s: q, pools and out must be 16-byte aligned", fn);
  const int32_t rows = num_seqs * num_kv_heads, group = num_q_heads / num_kv_heads;
  const pkv::SparseArgs a{selected, block_tables, seq_lens, num_seqs, num_kv_heads, max_selected, max_blocks,
                          num_blocks, block_size};
  if (sparse_by_cluster(dtype, max_selected)) {
    const double k = dtype == PKV_FP8_E4M3 ? k_scale : 1.0;
    const pkv::SparseDecodeArgs d{a, q, out, static_cast<float>(static_cast<double>(scale) * k * 1.4426950408889634),
                                  v_scale, g_stall_cta.load(std::memory_order_relaxed)};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool d128 = head_dim == 128;
    switch (dtype) {
      case PKV_BF16:
        return d128 ? launch_sparse_group<__nv_bfloat16, 128>(d, k_pool, v_pool, dtype, group, fn, s)
                    : launch_sparse_group<__nv_bfloat16, 64>(d, k_pool, v_pool, dtype, group, fn, s);
      case PKV_F16:
        return d128 ? launch_sparse_group<__half, 128>(d, k_pool, v_pool, dtype, group, fn, s)
                    : launch_sparse_group<__half, 64>(d, k_pool, v_pool, dtype, group, fn, s);
      default: return launch_sparse_group<pkv::E4m3, 128>(d, k_pool, v_pool, dtype, group, fn, s);
    }
  }
  if (!workspace) return fail(PKV_ERR_INVALID_ARG, "%s: NULL pointer", fn);
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return fail(PKV_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", fn);
  const SparseLayout w = sparse_layout(rows, group, head_dim, max_selected, block_size, kAutoPartitionTokens);
  if (workspace_bytes < w.total)
    return fail(PKV_ERR_INVALID_ARG, "%s: workspace %zu bytes < %zu needed", fn, workspace_bytes, w.total);
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  int32_t* tables = reinterpret_cast<int32_t*>(ws);
  int32_t* lens = reinterpret_cast<int32_t*>(ws + w.lens);
  cudaError_t e = launch_pdl(pkv::expand_selection_kernel, dim3(static_cast<unsigned>((int64_t(rows) + 7) / 8)),
                             dim3(256), 0, static_cast<cudaStream_t>(stream), a, tables, lens);
  if (e != cudaSuccess) return cuda_fail(e, fn);
  if (dtype == PKV_FP8_E4M3)
    return decode_fp8(fn, q, k_pool, v_pool, tables, lens, rows, group, 1, head_dim, num_blocks * num_kv_heads,
                      max_selected, block_size, scale, k_scale, v_scale, 0, ws + w.decode, workspace_bytes - w.decode,
                      out, nullptr, stream);
  return decode_16(fn, q, k_pool, v_pool, tables, lens, rows, group, 1, head_dim, num_blocks * num_kv_heads,
                   max_selected, block_size, scale, dtype, 0, ws + w.decode, workspace_bytes - w.decode, out, nullptr,
                   stream);
}

}  // namespace

extern "C" int pkv_block_bounds(const void* k_pool, const int32_t* block_tables, const int32_t* seq_lens,
                                const int32_t* new_tokens, int32_t max_new_tokens, int32_t num_seqs,
                                int32_t num_blocks, int32_t num_kv_heads, int32_t head_dim,
                                int32_t max_blocks_per_seq, int32_t block_size, int32_t dtype, void* bounds,
                                void* stream) {
  const char* fn = "pkv_block_bounds";
  NvtxRange nvtx_range(fn);
  int rc = check_sparse(fn, num_seqs, num_kv_heads, head_dim, num_blocks, max_blocks_per_seq, block_size, dtype);
  if (rc) return rc;
  if (max_new_tokens < 0 || (!new_tokens && max_new_tokens < 1))
    return fail(PKV_ERR_INVALID_ARG, "%s: max_new_tokens %d", fn, max_new_tokens);
  if (num_seqs == 0 || max_new_tokens == 0 || max_blocks_per_seq == 0) return pkv::ok();
  if (!k_pool || !block_tables || !seq_lens || !bounds) return fail(PKV_ERR_INVALID_ARG, "%s: NULL pointer", fn);
  if (!aligned16(k_pool) || !aligned16(bounds))
    return fail(PKV_ERR_INVALID_ARG, "%s: k_pool and bounds must be 16-byte aligned", fn);
  pkv::BoundsArgs a{};
  a.k_pool = k_pool;
  a.block_tables = block_tables;
  a.seq_lens = seq_lens;
  a.new_tokens = new_tokens;
  a.bounds = bounds;
  a.num_seqs = num_seqs;
  a.num_blocks = num_blocks;
  a.num_kv_heads = num_kv_heads;
  a.max_blocks = max_blocks_per_seq;
  a.block_size = block_size;
  a.max_new = max_new_tokens;
  // n tokens in a row touch at most (n + block_size - 2) / block_size + 1 blocks
  a.window = static_cast<int32_t>(
      std::min<int64_t>(max_blocks_per_seq, (int64_t(max_new_tokens) + block_size - 2) / block_size + 1));
  if (int64_t(num_seqs) * a.window * num_kv_heads > (int64_t(1) << 33))
    return fail(PKV_ERR_INVALID_ARG, "%s: too many blocks in one call", fn);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool d128 = head_dim == 128;
  cudaError_t e;
  switch (dtype) {
    case PKV_F32: e = d128 ? launch_bounds<float, 128>(a, s) : launch_bounds<float, 64>(a, s); break;
    case PKV_BF16: e = d128 ? launch_bounds<__nv_bfloat16, 128>(a, s) : launch_bounds<__nv_bfloat16, 64>(a, s); break;
    case PKV_F16: e = d128 ? launch_bounds<__half, 128>(a, s) : launch_bounds<__half, 64>(a, s); break;
    default: e = launch_bounds<pkv::E4m3, 128>(a, s);
  }
  if (e != cudaSuccess) return cuda_fail(e, fn);
  return pkv::ok();
}

extern "C" int pkv_select_workspace_size(int32_t num_seqs, int32_t num_kv_heads, int32_t max_blocks_per_seq,
                                         size_t* bytes) {
  const char* fn = "pkv_select_workspace_size";
  if (!bytes) return fail(PKV_ERR_INVALID_ARG, "%s: bytes is NULL", fn);
  if (num_seqs < 0 || num_kv_heads <= 0 || max_blocks_per_seq < 0 || max_blocks_per_seq > kMaxSelectBlocks ||
      int64_t(num_seqs) * num_kv_heads > (int64_t(1) << 24))
    return fail(PKV_ERR_INVALID_ARG, "%s: bad sizes", fn);
  *bytes = std::max<size_t>(256, select_layout(int64_t(num_seqs) * num_kv_heads, max_blocks_per_seq).total);
  return pkv::ok();
}

extern "C" int pkv_block_select(const void* q, const void* bounds, const int32_t* block_tables,
                                const int32_t* seq_lens, int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                int32_t head_dim, int32_t num_blocks, int32_t max_blocks_per_seq, int32_t block_size,
                                int32_t max_selected, int32_t n_first, int32_t n_last, int32_t dtype, void* workspace,
                                size_t workspace_bytes, int32_t* selected, void* stream) {
  const char* fn = "pkv_block_select";
  NvtxRange nvtx_range(fn);
  int rc = check_sparse(fn, num_seqs, num_kv_heads, head_dim, num_blocks, max_blocks_per_seq, block_size, dtype);
  if (rc) return rc;
  rc = check_group(fn, num_q_heads, num_kv_heads, false);
  if (rc) return rc;
  if (max_selected <= 0 || n_first < 0 || n_last < 0 || int64_t(n_first) + n_last > max_selected)
    return fail(PKV_ERR_INVALID_ARG, "%s: need max_selected >= 1 and n_first + n_last <= max_selected", fn);
  if (num_seqs == 0) return pkv::ok();
  if (!q || !bounds || !block_tables || !seq_lens || !workspace || !selected)
    return fail(PKV_ERR_INVALID_ARG, "%s: NULL pointer", fn);
  if (!aligned16(q) || !aligned16(bounds))
    return fail(PKV_ERR_INVALID_ARG, "%s: q and bounds must be 16-byte aligned", fn);
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return fail(PKV_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", fn);
  const int64_t rows = int64_t(num_seqs) * num_kv_heads;
  const SelectLayout w = select_layout(rows, max_blocks_per_seq);
  if (workspace_bytes < w.total)
    return fail(PKV_ERR_INVALID_ARG, "%s: workspace %zu bytes < %zu needed", fn, workspace_bytes, w.total);
  if (rows * ((max_blocks_per_seq + 15) / 16) > INT32_MAX)
    return fail(PKV_ERR_INVALID_ARG, "%s: too many blocks in one call", fn);
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  pkv::SelectArgs a{};
  a.q = q;
  a.bounds = bounds;
  a.block_tables = block_tables;
  a.seq_lens = seq_lens;
  a.scores = reinterpret_cast<float*>(ws);
  a.stats = reinterpret_cast<pkv::TileStats*>(ws + w.stats);
  a.fine = reinterpret_cast<uint64_t*>(ws + w.fine);
  a.selected = selected;
  a.num_seqs = num_seqs;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = num_kv_heads;
  a.num_blocks = num_blocks;
  a.max_blocks = max_blocks_per_seq;
  a.block_size = block_size;
  a.max_selected = max_selected;
  a.n_first = n_first;
  a.n_last = n_last;
  a.tiles = (max_blocks_per_seq + 15) / 16;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool d128 = head_dim == 128;
  switch (dtype) {
    case PKV_F32: return d128 ? launch_select_group<float, 128>(a, fn, s) : launch_select_group<float, 64>(a, fn, s);
    case PKV_BF16: return d128 ? launch_select_group<__nv_bfloat16, 128>(a, fn, s) : launch_select_group<__nv_bfloat16, 64>(a, fn, s);
    case PKV_F16: return d128 ? launch_select_group<__half, 128>(a, fn, s) : launch_select_group<__half, 64>(a, fn, s);
    default: return launch_select_group<pkv::E4m3, 128>(a, fn, s);
  }
}

extern "C" int pkv_sparse_workspace_size(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                         int32_t head_dim, int32_t max_selected, int32_t block_size, int32_t dtype,
                                         size_t* bytes) {
  const char* fn = "pkv_sparse_workspace_size";
  if (!bytes) return fail(PKV_ERR_INVALID_ARG, "%s: bytes is NULL", fn);
  int rc = check_sparse(fn, num_seqs, num_kv_heads, head_dim, 1, 0, block_size, dtype);
  if (rc) return rc;
  rc = check_group(fn, num_q_heads, num_kv_heads, dtype == PKV_F32);
  if (rc) return rc;
  if (max_selected <= 0 || int64_t(max_selected) * block_size > (int64_t(1) << 30))
    return fail(PKV_ERR_INVALID_ARG, "%s: max_selected %d", fn, max_selected);
  *bytes = sparse_by_cluster(dtype, max_selected)
               ? 0
               : sparse_layout(int64_t(num_seqs) * num_kv_heads, num_q_heads / num_kv_heads, head_dim, max_selected,
                               block_size, kAutoPartitionTokens).total;
  return pkv::ok();
}

extern "C" int pkv_paged_attention_decode_sparse(const void* q, const void* k_pool, const void* v_pool,
                                                 const int32_t* block_tables, const int32_t* seq_lens,
                                                 const int32_t* selected, int32_t max_selected, int32_t num_seqs,
                                                 int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                                 int32_t num_blocks, int32_t max_blocks_per_seq, int32_t block_size,
                                                 float scale, int32_t dtype, void* workspace, size_t workspace_bytes,
                                                 float* out, void* stream) {
  const char* fn = "pkv_paged_attention_decode_sparse";
  NvtxRange nvtx_range(fn);
  if (dtype == PKV_FP8_E4M3) return fail(PKV_ERR_UNSUPPORTED, "%s: e4m3 pools take the _fp8 form", fn);
  return sparse_decode(fn, q, k_pool, v_pool, block_tables, seq_lens, selected, max_selected, num_seqs, num_q_heads,
                       num_kv_heads, head_dim, num_blocks, max_blocks_per_seq, block_size, scale, dtype, 1.f, 1.f,
                       workspace, workspace_bytes, out, stream);
}

extern "C" int pkv_paged_attention_decode_sparse_fp8(const void* q, const void* k_pool, const void* v_pool,
                                                     const int32_t* block_tables, const int32_t* seq_lens,
                                                     const int32_t* selected, int32_t max_selected, int32_t num_seqs,
                                                     int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                                     int32_t num_blocks, int32_t max_blocks_per_seq,
                                                     int32_t block_size, float scale, float k_scale, float v_scale,
                                                     void* workspace, size_t workspace_bytes, float* out,
                                                     void* stream) {
  const char* fn = "pkv_paged_attention_decode_sparse_fp8";
  NvtxRange nvtx_range(fn);
  return sparse_decode(fn, q, k_pool, v_pool, block_tables, seq_lens, selected, max_selected, num_seqs, num_q_heads,
                       num_kv_heads, head_dim, num_blocks, max_blocks_per_seq, block_size, scale, PKV_FP8_E4M3, k_scale,
                       v_scale, workspace, workspace_bytes, out, stream);
}
