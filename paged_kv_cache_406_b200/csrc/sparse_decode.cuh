// Decode attention over selected blocks: for every sequence b and KV head g
// the softmax of q.K runs over the tokens of the blocks listed in
// selected[b][g][...] (ascending logical indices, -1 after the last) only.
#pragma once

#include <cuda.h>

#include "block_select.cuh"
#include "decode.cuh"
#include "device_common.cuh"

namespace pkv {

struct SparseArgs {
  const int32_t* selected;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  int32_t num_seqs, num_kv_heads, max_selected, max_blocks, num_blocks, block_size;
};

// The selection as a batch of its own: row (b, g) becomes a sequence with one
// KV head in a pool of num_blocks * num_kv_heads tiles, whose table lists the
// selected tiles.  One warp per row.  A list ends at the first entry that is
// negative, not above its predecessor or beyond the sequence; the latter two
// are recorded.
__global__ void __launch_bounds__(256) expand_selection_kernel(const SparseArgs a, int32_t* __restrict__ tables,
                                                               int32_t* __restrict__ lens) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (row >= static_cast<int64_t>(a.num_seqs) * a.num_kv_heads) return;
  const int b = static_cast<int>(row / a.num_kv_heads), g = static_cast<int>(row % a.num_kv_heads);
  const int L = a.seq_lens[b];
  int n = 0, last = -1;  // entries so far and the last of them
  if (L < 0 || L > a.max_blocks * a.block_size) {
    if (lane == 0) record_error(PKV_ERR_INVALID_ARG);
  } else {
    const int nblk = (L + a.block_size - 1) / a.block_size;
    const int32_t* sel = a.selected + row * a.max_selected;
    for (int i0 = 0; i0 < a.max_selected; i0 += 32) {
      const int i = i0 + lane;
      const int j = i < a.max_selected ? sel[i] : -1;
      int before = __shfl_up_sync(kFull, j, 1);
      if (lane == 0) before = last;
      const bool good = j >= 0 && j < nblk && j > before;
      const uint32_t bad = __ballot_sync(kFull, !good);
      const int end = bad ? __ffs(bad) - 1 : 32;
      if (lane == end && j >= 0) record_error(PKV_ERR_INVALID_ARG);
      if (lane < end) {
        int phys = a.block_tables[static_cast<int64_t>(b) * a.max_blocks + j];
        if (static_cast<unsigned>(phys) >= static_cast<unsigned>(a.num_blocks)) {
          record_error(PKV_ERR_BAD_BLOCK);
          phys = 0;
        }
        tables[row * a.max_selected + i] = phys * a.num_kv_heads + g;
      }
      n += end;
      if (end) last = __shfl_sync(kFull, j, end - 1);
      if (end < 32) break;
    }
    if (lane == 0) lens[row] = n == 0 ? 0 : (n - 1) * a.block_size + min(a.block_size, L - last * a.block_size);
    return;
  }
  if (lane == 0) lens[row] = 0;
}

// ---------------------------------------------------------------------------
// 16-bit and e4m3 pools: a cluster of CTAs per (sequence, KV head).
//
// Bytes bound it: the K and V rows of the selected blocks, read once.  All
// rows of a batch have about the same work and far less of it than dense
// decode's, so nothing is planned: the warps of the row's cluster take its
// 16-token chunks in turn, each with its own online softmax, and the cluster
// joins them through distributed shared memory.
//
// A warp streams its chunks through 16 KB of shared memory of its own (tensor
// map loads issued by its lane 0, 128-byte swizzle), so it waits for nothing
// but its own next chunk:
//     S[8 heads][16 tokens]   = Q[8 (of 16)][D] . K^T        (two 8-token tiles)
//     O^T[D][8 heads]        += V^T[D][16 tokens] . P^T[16][8]
// Lane (q, t) = (lane / 4, lane % 4) reads 16-byte pieces of K rows q and
// q + 8, which are B fragments of S in a channel order that Q's fragments
// share, and of V rows 2t, 2t + 1, 2t + 8, 2t + 9, whose halves exchanged
// (prmt) are A fragments of O^T in an order of channels undone at the end.
// S leaves each lane with head q at tokens 2t, 2t + 1, 2t + 8, 2t + 9: P's B
// fragments as they are.
//
// P enters as a sum of three bf16 values (24 bits at any size; weights are at
// most 1, since a bf16 value times more could leave 32 bits' range) or of two
// f16 ones.  f16 steps by 2^-24 however small a value is, so for f16 the unit of
// the weights follows the scores down as well as up: the largest weight of a
// lane's four tokens lies between 1 and 2^15, or, where the chunk's tokens
// differ by more, its largest weight at 2^15.  A weight keeps 22 bits, or 2^-25
// of its lane's largest, or 2^-40 of its chunk's, down to 2^-60 of the row's
// largest.  1439 tokens e^-12, e^-15 and e^-18 below a sink token of value 0: the
// output is off by 5e-7, 6e-7 and 3e-6 of itself, against each warp's largest
// alone 2e-4, 5e-3 and 8e-2 (the sink's warp lost its other tokens).  The unit is
// a whole power of two, so moving it is exact.
//
// 512 rows of 64 bf16 blocks of 16 tokens (268 MB): 47.7 us, 5.6 TB/s; the
// dense kernels on the selection as a batch of its own take 52 to 56, loads
// straight into registers 60 to 66 (a warp then waits for its own loads).  Of
// e4m3 blocks (135 MB): 37.4 us, 3.6 TB/s, bound by the instructions that widen
// K and V.  A row alone costs 6 us: the list, a chunk, the join.
// ---------------------------------------------------------------------------
constexpr int kSparseList = 1024;   // most selected blocks (they lie in shared memory)
constexpr int kSparseCluster = 8;
// Warps of a CTA: three where there are many rows (four CTAs an SM, so that 592
// rows run at once and end together), eight where there are few.
constexpr int kSparseFewWarps = 3, kSparseManyWarps = 8;

template <typename T, int D, int G, int kWarps>
struct SparseSmem {
  static constexpr int kRow = D * static_cast<int>(sizeof(T));  // bytes of a token
  static constexpr int kTile = 16 * kRow;                       // K (or V) of a chunk
  static constexpr int kStage = 2 * kTile;
  static constexpr int kStages = 16 * 1024 / kStage;            // 2 or 4
  static constexpr int kRec = (G * D + 2 * G + 3) / 4 * 4;      // O, m, l of a warp or a CTA; 16-byte aligned
  static constexpr int kRing = kWarps * kStages * kStage;       // the records take its place at the end
  static constexpr int kRecBytes = kWarps * kRec * 4;
  static constexpr int kBytes = 1024 + (kRing > kRecBytes ? kRing : kRecBytes);  // 1024: the swizzle's alignment
};

struct SparseDecodeArgs {
  SparseArgs s;
  const void* q;
  float* out;
  float scale_log2, v_scale;
  // Test support for the bounded waits (pkv_debug_stall_decode): the warps of
  // CTA `stall_cta` leave out their first chunk's copies.  < 0 in normal calls.
  int32_t stall_cta;
};

// 2^e of a whole e; 0 below 2^-126.
__device__ __forceinline__ float exp2_whole(float e) {
  return __int_as_float((__float2int_rn(fminf(fmaxf(e, -127.f), 127.f)) + 127) << 23);
}

template <typename T, int D, int G, int kWarps>
__global__ void __launch_bounds__(kWarps * 32, kWarps == kSparseFewWarps ? 4 : 1)
    sparse_decode_kernel(const SparseDecodeArgs a, const __grid_constant__ CUtensorMap kmap,
                         const __grid_constant__ CUtensorMap vmap) {
  using Q = typename QueryOf<T>::type;
  using Smem = SparseSmem<T, D, G, kWarps>;
  constexpr bool kFp8 = sizeof(T) == 1;
  constexpr int kThreads = kWarps * 32, kRow = Smem::kRow, kNS = Smem::kStages, kRec = Smem::kRec;
  constexpr int kKP = kRow / 64, kVP = kRow / 128;       // pieces of a K row (four lanes) and a V row (eight lanes)
  constexpr int kSteps = kFp8 ? 4 : 2;                   // mma steps of a K piece
  constexpr int kTiles = kFp8 ? 8 : 4;                   // channel pairs of a V piece
  constexpr bool kBf16 = std::is_same_v<Q, __nv_bfloat16>;
  constexpr int kTerms = kBf16 ? 3 : 2;
  extern __shared__ unsigned char sparse_raw[];
  __shared__ int32_t list[kSparseList];
  __shared__ int32_t first_bad;
  __shared__ int32_t abort_word;
  __shared__ __align__(8) uint64_t full[kWarps][kNS];
  unsigned char* ring = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(sparse_raw) + 1023) & ~uintptr_t(1023));
  float* rec = reinterpret_cast<float*>(ring);  // [kWarps][kRec], once the ring is done with
  volatile int* abort_flag = &abort_word;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  uint32_t rank, ctas;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
  const int64_t row = blockIdx.x / ctas;
  const int b = static_cast<int>(row / a.s.num_kv_heads), g = static_cast<int>(row - static_cast<int64_t>(b) * a.s.num_kv_heads);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gq = lane >> 2, tq = lane & 3;
  const int bs = a.s.block_size, bs_shift = bs == 8 ? 3 : (bs == 16 ? 4 : 5), K = a.s.max_selected;

  // ---- the tiles of the selected blocks ----
  const int32_t* sel = a.s.selected + row * K;
  const int L = a.s.seq_lens[b];
  const bool fits = L >= 0 && L <= a.s.max_blocks * bs;
  const int nblk = fits ? (L + bs - 1) >> bs_shift : 0;
  if (tid == 0) {
    first_bad = K;
    abort_word = 0;
    if (!fits && rank == 0) record_error(PKV_ERR_INVALID_ARG);
    for (int w = 0; w < kWarps; ++w)
      for (int i = 0; i < kNS; ++i) mbar_init(smem_addr(&full[w][i]), 1);
    fence_mbar_init();
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&vmap);
  }
  // A fragments of Q: row gq is head gq (zero from G on, as are rows 8 .. 15)
  uint32_t qa[kKP][kSteps][2];
#pragma unroll
  for (int i = 0; i < kKP; ++i)
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      uint2 w = make_uint2(0, 0);
      if (gq < G)
        w = *reinterpret_cast<const uint2*>(static_cast<const Q*>(a.q) + (row * G + gq) * D + (4 * i + tq) * 2 * kSteps * 2 + 4 * s);
      qa[i][s][0] = w.x;
      qa[i][s][1] = w.y;
    }
  __syncthreads();
  for (int i = tid; i < K; i += kThreads) {
    const int j = sel[i], before = i ? sel[i - 1] : -1;
    if (j >= 0 && j < nblk && j > before) {
      int phys = a.s.block_tables[static_cast<int64_t>(b) * a.s.max_blocks + j];
      if (static_cast<unsigned>(phys) >= static_cast<unsigned>(a.s.num_blocks)) {
        phys = -1;  // recorded below if the list reaches it
      }
      list[i] = phys;
    } else {
      atomicMin(&first_bad, i);
    }
  }
  __syncthreads();
  const int n = first_bad;  // the list's length
  if (rank == 0 && tid == 0 && n < K && sel[n] >= 0 && fits) record_error(PKV_ERR_INVALID_ARG);
  for (int i = tid; i < n; i += kThreads) {
    if (list[i] < 0) {
      record_error(PKV_ERR_BAD_BLOCK);
      list[i] = 0;
    }
  }
  __syncthreads();
  const int tokens = n ? ((n - 1) << bs_shift) + min(bs, L - (sel[n - 1] << bs_shift)) : 0;
  const int chunks = (tokens + 15) >> 4;

  // ---- the warp's ring ----
  // A tile lies as the tensor map's boxes of `box` rows: [box][128-byte half][row]
  // [128 B], 16-byte pieces exchanged by the row's number mod 8.
  const int box = min(bs, 16), step = static_cast<int>(ctas) * kWarps, c_first = static_cast<int>(rank) * kWarps + warp;
  const uint32_t ring_s = smem_addr(ring) + warp * kNS * Smem::kStage;
  const uint64_t policy = l2_evict_first_policy();
  auto issue = [&](int c, int stage) {  // lane 0
    const uint32_t bar = smem_addr(&full[warp][stage]), dst = ring_s + stage * Smem::kStage;
    const int boxes = bs == 8 ? min(2, n - 2 * c) : 1;
    mbar_arrive_expect_tx(bar, boxes * 2 * box * kRow);
    for (int i = 0; i < boxes; ++i) {
      const int token = c * 16 + i * 8;
      const int y = (list[token >> bs_shift] * a.s.num_kv_heads + g) * bs + (token & (bs - 1));
      tma_load_3d(dst + i * box * kRow, &kmap, 0, y, 0, bar, policy);
      tma_load_3d(dst + Smem::kTile + i * box * kRow, &vmap, 0, y, 0, bar, policy);
    }
  };
  // 16 bytes at byte `at` of row r of a tile
  auto piece = [&](uint32_t tile, int r, int at) {
    const int rr = r & (box - 1);
    const uint32_t addr = tile + (r - rr) * kRow + ((at >> 7) * box + rr) * 128 + ((((at >> 4) & 7) ^ (rr & 7)) << 4);
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
  };
  if (lane == 0) {
    for (int i = 0; i < kNS; ++i)
      if (c_first + i * step < chunks && (i > 0 || a.stall_cta != static_cast<int>(blockIdx.x)))
        issue(c_first + i * step, i);
  }

  float acc[kVP][kTiles][4];
#pragma unroll
  for (int i = 0; i < kVP; ++i)
#pragma unroll
    for (int t = 0; t < kTiles; ++t) acc[i][t][0] = acc[i][t][1] = acc[i][t][2] = acc[i][t][3] = 0.f;
  float m = kLowest, l = 0.f, top = kLowest;  // of head gq; m is whole; top: the largest score where m was moved
  int stage = 0;
  uint32_t phase = 0;
  for (int c = c_first; c < chunks; c += step) {
    const bool landed = __all_sync(kFull, mbar_wait(smem_addr(&full[warp][stage]), phase, abort_flag));
    if (!landed) {  // give up, after the copies that are still on their way
      if (lane == 0) {
        record_error(PKV_ERR_DEVICE_TIMEOUT);
        *abort_flag = 1;
        for (int i = 0; i < kNS && c + i * step < chunks; ++i) {
          const int st = (stage + i) % kNS;
          mbar_drain(smem_addr(&full[warp][st]), st < stage ? phase ^ 1 : phase);
        }
      }
      break;
    }
    const uint32_t ktile = ring_s + stage * Smem::kStage, vtile = ktile + Smem::kTile;
    // ---- scores ----
    float s[2][4] = {};
#pragma unroll
    for (int i = 0; i < kKP; ++i)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint4 x = piece(ktile, gq + 8 * r, i * 64 + tq * 16);
        const uint32_t v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int t = 0; t < kSteps; ++t) {
          const uint32_t qf[4] = {qa[i][t][0], 0u, qa[i][t][1], 0u};
          if constexpr (kFp8) mma_16816<Q>(s[r], qf, e4m3x2_to_f16x2(v[t]), e4m3x2_to_f16x2(v[t] >> 16));
          else mma_16816<Q>(s[r], qf, v[2 * t], v[2 * t + 1]);
        }
      }
    const int nv = tokens - c * 16;  // valid tokens from the chunk's first
    float x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int token = 2 * tq + (k & 1) + 8 * (k >> 1);
      x[k] = token < nv ? s[k >> 1][k & 1] * a.scale_log2 : -INFINITY;
    }
    // ---- online softmax: weights, sums and outputs in units of 2^m ----
    float bm = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
    const bool stay = kBf16 ? bm <= m + kRescaleThreshold : bm >= m && bm <= __fadd_rd(m, 15.f);
    if (!__all_sync(kFull, stay)) {
      const float own = bm;
      bm = fmaxf(bm, __shfl_xor_sync(kFull, bm, 1));
      bm = ceilf(fmaxf(fmaxf(bm, __shfl_xor_sync(kFull, bm, 2)), kLowest));  // of head gq
      float nm;
      if constexpr (kBf16) {
        nm = fmaxf(m, bm);
      } else {
        top = fmaxf(top, bm);
        // some lane far below the chunk's largest: as many bits for it as there are
        const float up = __any_sync(kFull, own < bm - 7.f) ? -15.f : -7.f;
        nm = fmaxf(__fadd_ru(bm, up), top - 60.f);
      }
      const float f = exp2_whole(m - nm);
      m = nm;
      l *= f;
      const float f0 = __shfl_sync(kFull, f, 8 * tq), f1 = __shfl_sync(kFull, f, 8 * tq + 4);  // heads 2 tq, 2 tq + 1
#pragma unroll
      for (int i = 0; i < kVP; ++i)
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          acc[i][t][0] *= f0;
          acc[i][t][2] *= f0;
          acc[i][t][1] *= f1;
          acc[i][t][3] *= f1;
        }
    }
    uint32_t pb[kTerms][2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float p0 = fast_exp2(x[2 * r] - m), p1 = fast_exp2(x[2 * r + 1] - m);
      if constexpr (kBf16) {  // at most 2^kRescaleThreshold so far
        p0 *= 0.00390625f;
        p1 *= 0.00390625f;
      }
      l += p0 + p1;
#pragma unroll
      for (int t = 0; t < kTerms; ++t) {
        Chunk<Q, 2> h;
        h.e[0] = narrow1<Q>(p0);
        h.e[1] = narrow1<Q>(p1);
        p0 -= widen1<Q>(h.e[0]);
        p1 -= widen1<Q>(h.e[1]);
        pb[t][r] = h.raw;
      }
    }
    // ---- O^T += V^T . P^T ----
#pragma unroll
    for (int i = 0; i < kVP; ++i) {
      uint32_t w[4][kTiles];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int token = 2 * tq + (r & 1) + 8 * (r >> 1);
        uint4 y = piece(vtile, token, i * 128 + gq * 16);
        if (token >= nv) y = make_uint4(0, 0, 0, 0);  // whatever lies behind the last token
        const uint32_t v[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if constexpr (kFp8) {
            w[r][2 * k] = e4m3x2_to_f16x2(v[k]);
            w[r][2 * k + 1] = e4m3x2_to_f16x2(v[k] >> 16);
          } else {
            w[r][k] = v[k];
          }
        }
      }
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
        // row q: channel 2 t of the piece, row q + 8: channel 2 t + 1
        const uint32_t f[4] = {__byte_perm(w[0][t], w[1][t], 0x5410), __byte_perm(w[0][t], w[1][t], 0x7632),
                               __byte_perm(w[2][t], w[3][t], 0x5410), __byte_perm(w[2][t], w[3][t], 0x7632)};
        // A chunk's products are summed by themselves, the small terms first:
        // the tensor cores drop the bits of a sum that its largest part
        // pushes out, and a running sum would lose some at every chunk.
        float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = kTerms - 1; k >= 0; --k) mma_16816<Q>(o, f, pb[k][0], pb[k][1]);
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[i][t][k] += o[k];
      }
    }
    __syncwarp();  // every lane has read the stage
    if (lane == 0 && c + kNS * step < chunks) issue(c + kNS * step, stage);
    if (++stage == kNS) {
      stage = 0;
      phase ^= 1;
    }
  }

  // ---- join the warps ----
  l += __shfl_xor_sync(kFull, l, 1);
  l += __shfl_xor_sync(kFull, l, 2);
  __syncthreads();  // the ring's place is free
  float* mine = rec + warp * kRec;
#pragma unroll
  for (int i = 0; i < kVP; ++i)
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      const int d = (8 * i + gq) * 2 * kTiles + 2 * t;
#pragma unroll
      for (int x = 0; x < 2; ++x)
        if (2 * tq + x < G)
          *reinterpret_cast<float2*>(mine + (2 * tq + x) * D + d) = make_float2(acc[i][t][x], acc[i][t][2 + x]);
    }
  if (tq == 0 && gq < G) {
    mine[G * D + gq] = m;
    mine[G * D + G + gq] = l;
  }
  __syncthreads();
  // the CTA's record takes the place of warp 0's: each thread rewrites only what it alone reads
  float mh[kWarps];
  auto factors = [&](int h) {
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, rec[w * kRec + G * D + h]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mh[w] = fast_exp2(rec[w * kRec + G * D + h] - top);
    return top;
  };
  for (int e = tid * 4; e < G * D; e += kThreads * 4) {
    factors(e / D);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float4 y = *reinterpret_cast<const float4*>(&rec[w * kRec + e]);
      o.x += mh[w] * y.x;
      o.y += mh[w] * y.y;
      o.z += mh[w] * y.z;
      o.w += mh[w] * y.w;
    }
    *reinterpret_cast<float4*>(&rec[e]) = o;
  }
  float cta_m = 0.f, cta_l = 0.f;
  if (tid < G) {
    cta_m = factors(tid);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) cta_l += mh[w] * rec[w * kRec + G * D + G + tid];
  }
  __syncthreads();
  if (tid < G) {
    rec[G * D + tid] = cta_m;
    rec[G * D + G + tid] = cta_l;
  }

  // ---- join the CTAs: each finishes a share of the outputs ----
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  auto remote = [&](const float* p, uint32_t r) {
    uint32_t addr;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_addr(p)), "r"(r));
    return addr;
  };
  for (int e = (static_cast<int>(rank) * kThreads + tid) * 4; e < G * D; e += static_cast<int>(ctas) * kThreads * 4) {
    const int h = e / D;
    float cm[kSparseCluster], top = -INFINITY, den = 0.f;
#pragma unroll
    for (int r = 0; r < kSparseCluster; ++r) {
      cm[r] = -INFINITY;
      if (r < static_cast<int>(ctas))
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(cm[r]) : "r"(remote(&rec[G * D + h], r)) : "memory");
      top = fmaxf(top, cm[r]);
    }
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int r = 0; r < kSparseCluster; ++r) {
      if (r < static_cast<int>(ctas)) {
        float cl;
        float4 y;
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(cl) : "r"(remote(&rec[G * D + G + h], r)) : "memory");
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(y.x), "=f"(y.y), "=f"(y.z), "=f"(y.w)
                     : "r"(remote(&rec[e], r))
                     : "memory");
        const float f = fast_exp2(cm[r] - top);
        den += f * cl;
        o.x += f * y.x;
        o.y += f * y.y;
        o.z += f * y.z;
        o.w += f * y.w;
      }
    }
    const float inv = den == 0.f ? 0.f : a.v_scale / den;
    *reinterpret_cast<float4*>(a.out + row * G * D + e) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
  }
  // no CTA leaves while another reads its record
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

}  // namespace pkv
