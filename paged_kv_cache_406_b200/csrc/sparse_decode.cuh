// Decode attention over selected blocks: for every sequence b and KV head g
// the softmax of q.K runs over the tokens of the blocks listed in
// selected[b][g][...] (ascending logical indices, -1 after the last) only.
#pragma once

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

}  // namespace pkv
