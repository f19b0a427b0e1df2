// Page accounting and forks: arguments shared by the host side and s4kv_pages.cu.
#pragma once

#include "s4kv_common.cuh"

namespace s4kv {

constexpr int kMaxPageJobs = 4096;    // sequences of one call
constexpr int kMaxPageRows = 65536;   // rows of a block table

struct PageArgs {
  int* status;
  int* refs;                // [num_pages]: table entries that name the page
  int* table;               // [rows][bt_stride]
  const int* slot_ids;      // take, release: a sequence's row, or null (its index)
  const int* from;          // take: lengths before; release: first tokens; fork: source rows
  const int* to;            // take: lengths after; release: last tokens; fork: new rows
  const int* seq_lens;      // fork
  int* taken;
  int bt_stride, rows, n, num_pages;
  // fork
  char* pool_layers;        // the first layer's region
  int* lens;                // [layers][max_slots][H]
  size_t layer_stride, kring_offset, vring_offset, kring_slot, vring_slot, kring_head, vring_head, page_bytes;
  int layers, H, R, max_slots, bits;
  int pages_at_most;        // pages of a fork whose contents may have to be copied
};

cudaError_t launch_take(const PageArgs& a, cudaStream_t st);
cudaError_t launch_release(const PageArgs& a, cudaStream_t st);
cudaError_t launch_fork(const PageArgs& a, cudaStream_t st);

// What of a sequence of T tokens sits where, by page format: pages below `done` are never written
// again, pages below `held` hold something; 16-bit rows 0 .. krows - 1 and 0 .. vrows - 1 of the rings.
struct Held {
  int done, held, krows, vrows;
};
__host__ __device__ inline Held held_of(int bits, int T, int R) {
  Held x;
  if (bits == 8) return Held{T / kP, (T + kP - 1) / kP, 0, 0};
  if (bits == S4KV_BITS_INT8) return Held{T / kP, T / kP, T % kP, T % kP};
  const int Tk = T / kG * kG, Tv = T > R ? T - R : 0;
  x.done = (Tk < Tv ? Tk : Tv) / kP;
  x.held = ((Tk < Tv ? Tv : Tk) + kP - 1) / kP;
  x.krows = T - Tk;
  x.vrows = T < R ? T : R;
  return x;
}

}  // namespace s4kv
