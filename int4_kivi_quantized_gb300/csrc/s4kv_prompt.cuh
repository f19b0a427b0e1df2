// Prompt attention (s4kv_prompt_attention): what its launches share. The first restores the
// cached tokens into tiles of matrix operands (s4kv_tiles.cu), the second attends
// (s4kv_prompt.cu), a third combines where the cache's length was split.
//
// Workspace: tiles (by kv tile of the call and kv head, 64 KB: 128 tokens' keys, then values, as
// f16 in the image that the tensor cores read), one bit a token (its value row is not finite),
// and the partial outputs of a split call.
#pragma once

#include "s4kv_score.cuh"

namespace s4kv {

constexpr int kQRows = 256;          // (token, head) rows of a CTA: two tiles of 128
constexpr int kKvTile = 128;         // cached tokens of a tile
constexpr int kTileBytes = kKvTile * kD * 2;
constexpr int kMaxSplits = 16;

struct PromptArgs {
  const char* pages;
  const char* kring;
  const char* vring;
  const int* lens;
  int* status;
  const int* block_table;
  const int* seq_lens;
  const int* slot_ids;
  const int* cu_q;
  const uint16_t* q;
  void* out;
  const float* fp8_scale;
  ScoreForm form;
  char* tiles;
  uint32_t* bad;            // [kv tile][H][4]: a bit a token
  float* part;              // [q tile][H][split][256][128], then [q tile][H][split][256][2]
  long long kring_slot, kring_head, vring_slot, vring_head;
  long long wait_ns;
  float sm_scale;
  int bt_stride, n, num_q, Hq, H, g, R, num_pages, max_slots, dtype, out_dtype, bits, max_seq_len;
  int kv_tiles, q_tiles;    // at most, of the call
  int kv_grid;              // kv tiles that a window leaves, at most
  int splits;
};

cudaError_t launch_tiles(const PromptArgs& a, cudaStream_t st);
cudaError_t launch_prompt(const PromptArgs& a, cudaStream_t st);

namespace {

// A sequence's tiles. Rows of queries: whole or partly filled tiles of its own; cached tokens: the
// same, for a sequence that has queries and a length that can be (others have none).
__device__ __forceinline__ int q_tiles_of(const PromptArgs& a, int m) {
  return m > 0 ? static_cast<int>((static_cast<long long>(m) * a.g + kQRows - 1) / kQRows) : 0;
}
// The kv tiles of a sequence that some query of its chunk may see: the sinks' [0, sinks) and [first, end).
struct KvRange {
  int sinks, first, end;
  __device__ __forceinline__ int count() const { return sinks + end - first; }
  __device__ __forceinline__ int at(int j) const { return j < sinks ? j : j - (first - sinks); }   // place of tile j in the workspace
  __device__ __forceinline__ int tile(int i) const { return i < sinks ? i : first + i - sinks; }   // and the other way
};
__device__ __forceinline__ KvRange kv_range(const PromptArgs& a, int m, int T) {
  KvRange r;
  r.end = (T - 1) / kKvTile + 1;
  r.sinks = min(a.form.sinks / kKvTile + (a.form.sinks % kKvTile != 0), r.end);
  r.first = max(r.sinks, max(0, T - m - a.form.window + 1) / kKvTile);
  return r;
}
__device__ __forceinline__ int kv_tiles_of(const PromptArgs& a, int m, int T) {
  return m > 0 && T >= m && T <= a.max_seq_len ? kv_range(a, m, T).count() : 0;
}

struct Place {
  int b, tile, kv0;         // sequence, tile within it (of kv tiles: place among those it has), its first kv tile of the call
  int cu0, m, T;            // its first row, its queries, its length
};
enum { kFound = 0, kNowhere = 1, kMalformed = 2 };

// Which sequence tile `idx` of the call belongs to, counting query tiles or kv tiles. Every
// thread of a CTA of `THREADS` calls it. kMalformed: cu_q is not what it should be.
template <int THREADS, bool BY_Q>
__device__ int find_tile(const PromptArgs& a, int idx, Place& place) {
  constexpr int W = THREADS / 32;
  __shared__ int tot[2][W];
  __shared__ Place found;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // (the attention kernel looks while the launch before it still runs, and so past the first cache)
  auto look = [](const int* x) { return BY_Q ? __ldcg(x) : *x; };
  if (a.n <= 32) {   // a sequence a lane, every warp for itself
    const int b = lane, c0 = b < a.n ? look(a.cu_q + b) : 0, c1 = b < a.n ? look(a.cu_q + b + 1) : 0, T = b < a.n ? look(a.seq_lens + b) : 0;
    const bool wrong = c0 < 0 || c1 < c0 || c1 > a.num_q || (b == 0 && c0 != 0) || (b == a.n - 1 && c1 != a.num_q);
    if (__any_sync(0xffffffffu, wrong)) return kMalformed;
    const int m = c1 - c0, qt = q_tiles_of(a, m), kt = kv_tiles_of(a, m, T);
    int q = qt, k = kt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, q, o), z = __shfl_up_sync(0xffffffffu, k, o);
      if (lane >= o) {
        q += y;
        k += z;
      }
    }
    const int first = BY_Q ? q - qt : k - kt;
    const unsigned here = __ballot_sync(0xffffffffu, idx >= first && idx - first < (BY_Q ? qt : kt));
    if (!here) return kNowhere;
    const int l = __ffs(here) - 1;
    place = Place{l, idx - __shfl_sync(0xffffffffu, first, l), __shfl_sync(0xffffffffu, k - kt, l), __shfl_sync(0xffffffffu, c0, l),
                  __shfl_sync(0xffffffffu, m, l), __shfl_sync(0xffffffffu, T, l)};
    return kFound;
  }
  int bad = 0, carry_q = 0, carry_k = 0;
  if (tid == 0) {
    bad = look(a.cu_q) != 0 || look(a.cu_q + a.n) != a.num_q;
    found.b = -1;
  }
  for (int base = 0; base < a.n; base += THREADS) {
    const int b = base + tid;
    int qt = 0, kt = 0, c0 = 0, m = 0, T = 0;
    if (b < a.n) {
      const int c1 = look(a.cu_q + b + 1);
      c0 = look(a.cu_q + b);
      T = look(a.seq_lens + b);
      m = c1 - c0;
      if (c0 < 0 || c1 < c0 || c1 > a.num_q) {
        bad = 1;
      } else {
        qt = q_tiles_of(a, m);
        kt = kv_tiles_of(a, m, T);
      }
    }
    int q = qt, k = kt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, q, o), z = __shfl_up_sync(0xffffffffu, k, o);
      if (lane >= o) {
        q += y;
        k += z;
      }
    }
    if (lane == 31) {
      tot[0][warp] = q;
      tot[1][warp] = k;
    }
    __syncthreads();
    int q0 = carry_q, k0 = carry_k;
    for (int w = 0; w < W; ++w) {
      if (w < warp) {
        q0 += tot[0][w];
        k0 += tot[1][w];
      }
      carry_q += tot[0][w];
      carry_k += tot[1][w];
    }
    q0 += q - qt;
    k0 += k - kt;
    const int first = BY_Q ? q0 : k0, count = BY_Q ? qt : kt;
    if (idx >= first && idx - first < count) found = Place{b, idx - first, k0, c0, m, T};
    __syncthreads();
  }
  if (__syncthreads_or(bad)) return kMalformed;
  place = found;
  return place.b >= 0 ? kFound : kNowhere;
}

// Why a sequence's part of the call cannot be done, 0 if it can; `arg` goes with it.
__device__ __forceinline__ int refused(const PromptArgs& a, const Place& p, int slot, int h, int& arg) {
  const int m = p.m, T = p.T;
  arg = p.b;
  if (slot < 0 || slot >= a.max_slots) {
    arg = slot;
    return S4KV_DEV_BAD_SLOT;
  }
  if (T < m || T > a.max_seq_len || __ldcg(a.lens + static_cast<long long>(slot) * a.H + h) != T) return S4KV_DEV_BAD_LENGTH;
  if (static_cast<long long>(a.bt_stride) * kP < T) return S4KV_DEV_BAD_TABLE;
  // more tokens in all than the caller said there are
  if (static_cast<long long>(p.kv0) + kv_tiles_of(a, m, T) > a.kv_tiles) return S4KV_DEV_BAD_LENGTH;
  return 0;
}

}  // namespace
}  // namespace s4kv
