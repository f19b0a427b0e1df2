// The first launch of prompt attention: every cached token that a chunk may see, restored from
// its page or ring into tiles of matrix operands.
//
// A tile is 128 tokens of one kv head, keys then values, f16, each as two halves of 64 channels
// of 128 rows (tokens) of 128 bytes whose 16-byte chunks c sit at c xor (row mod 8): the image
// that tcgen05 reads, as a K-major operand (keys) and as an MN-major one (values), so the attention
// kernel fetches a tensor's tile with one bulk copy. f16 keeps 11 bits of a restored value
// where the caches' bf16 would keep 8: a key's rounding then moves a score by 2^-11 of its
// terms at most. FP8 codes are exact in f16 and stay codes, at any scale. Values beyond f16's range become
// infinities; a value row with an element that is not finite (then) is stored as zeros where it is not and gets
// a bit, so that queries which do not see it never meet it.
//
// A CTA takes one tensor of a tile, a warp a page of it (of a key group on KIVI pages, whose metadata
// lie in two pages' records). 64 KB are written for every 8 to 17 KB read, and most of them stay in
// the L2 cache for the attention kernel. Measured (cold caches): 4 sequences behind a window of 4096, 2 bits, 8 kv
// heads, 74 MB of tiles 22 us, 3.4 TB/s; 8 INT8 sequences of 2048 to 8192, 168 MB 48 us, 3.5
// TB/s; one 4-bit prompt of 2048 8 us; 32768 tokens of 4 heads, 64 MB 22 us. The issue slots are 53 to 65%
// busy: what bounds it is a warp's few hundred instructions for 2048 elements and the chain lengths ->
// table -> record in front of them. Four CTAs an SM (64 registers) 59.6 us for the 2-bit call, three 61.7,
// as many with the table read behind the length check 63.6. Two pages a warp in CTAs of four warps spill
// or lose the occupancy: 62 to 67.

#include "s4kv_prompt.cuh"
#include "s4kv_restore.cuh"

namespace s4kv {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;

// Eight channels of row r0 + token of a tile's tensor. bits: of the tokens whose rows are not
// finite (values), or null (keys).
struct TileRows {
  char* tile;
  int r0;
  uint32_t* bits;
  __device__ __forceinline__ void operator()(int token, int c, const float (&y)[8]) const {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 x = __floats2half2_rn(y[2 * i], y[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&x);
    }
    const int r = r0 + token;
    if (bits) {
      // what is finite is a zero times zero
      __half2 z = __floats2half2_rn(0.0f, 0.0f);
      const __half2 zero = z;
#pragma unroll
      for (int i = 0; i < 4; ++i) z = __hfma2(*reinterpret_cast<const __half2*>(&w[i]), zero, z);
      if (*reinterpret_cast<const uint32_t*>(&z) & 0x7fff7fffu) {
        *bits |= 1u << (r & (kP - 1));
        w[0] = w[1] = w[2] = w[3] = 0u;
      }
    }
    store(c, r, make_uint4(w[0], w[1], w[2], w[3]));
  }
  __device__ __forceinline__ void store(int c, int r, uint4 w) const {
    *reinterpret_cast<uint4*>(tile + (c >> 3) * (kTileBytes / 2) + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = w;
  }
  // zeros in rows r0 + lo .. r0 + hi - 1
  __device__ __forceinline__ void clear(int lo, int hi) const {
    const int lane = threadIdx.x & 31;
    for (int t = lo + (lane >> 4); t < hi; t += 2) store(lane & 15, r0 + t, make_uint4(0u, 0u, 0u, 0u));
  }
};

template <int FMT>
__global__ void __launch_bounds__(kThreads, 4) tiles_kernel(PromptArgs a) {
  stream_wait();
  // the attention kernel may start: it waits for this one where it needs the tiles
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  Place p;
  const int h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool values = blockIdx.z;
  const int where = find_tile<kThreads, false>(a, blockIdx.x, p);
  if (where == kMalformed && blockIdx.x == 0 && h == 0 && !values && threadIdx.x == 0)
    report(a.status, S4KV_ERR_DEVICE, S4KV_DEV_BAD_CU, a.n);
  if (where != kFound) return;
  const int m = p.m, T = p.T, slot = a.slot_ids ? a.slot_ids[p.b] : p.b;
  const int tp = kv_range(a, m, T).tile(p.tile) * kKvTile + kP * warp;   // this warp's 16 tokens
  const long long at = (static_cast<long long>(p.kv0) + p.tile) * a.H + h;
  uint32_t bits = 0;
  const TileRows rows{a.tiles + (2 * at + values) * kTileBytes, kP * warp, values ? &bits : nullptr};
  const int* bt = a.block_table + static_cast<long long>(p.b) * a.bt_stride;
  const int Tk = FMT == 8 ? T : FMT == kI8 ? T / kP * kP : T & ~(kG - 1);
  const int Tv = FMT == 8 ? T : FMT == kI8 ? Tk : max(0, T - a.R);
  const int quant = values ? Tv : Tk, mod = FMT == kI8 ? kP : values ? a.R : kG;
  const uint16_t* ring = values ? reinterpret_cast<const uint16_t*>(a.vring) + slot * a.vring_slot + h * a.vring_head
                                : reinterpret_cast<const uint16_t*>(a.kring) + slot * a.kring_slot + h * a.kring_head;
  // A tile may reach past the tokens that some query sees (those from `low` on, and the sinks), to pages that the
  // sequence has given back: zeros, and the table is not looked at.
  const int low = max(0, T - m - a.form.window + 1);
  const bool seen = tp < a.form.sinks || tp + kP > low;
  const int end = seen ? min(max(T - tp, 0), kP) : 0;   // tokens [0, end) of this page are there
  const int held = min(max(quant - tp, 0), end);      // [0, held) in its record
  // the table's entries, on their way while the sequence is checked
  const bool group = !kByte<FMT> && !values;   // half of a key group: both its pages
  const int page = tp / kP;
  int pp[2] = {-1, -1};
  if (held > 0 && static_cast<long long>(a.bt_stride) * kP >= T) {
    pp[0] = bt[group ? page & ~1 : page];
    pp[1] = group ? bt[page | 1] : pp[0];
  }
  int arg;
  if (refused(a, p, slot, h, arg)) return;   // (the attention kernel says so)
  auto record = [&](int pp) -> const char* {   // null (reported) outside the pool
    if (pp >= 0 && pp < a.num_pages) return a.pages + (static_cast<long long>(pp) * a.H + h) * Rec<FMT>::kBytes;
    if (lane == 0) report(a.status, S4KV_ERR_DEVICE, S4KV_DEV_BAD_PAGE, pp);
    return nullptr;
  };
  if (held > 0) {
    if (group) {
      if constexpr (!kByte<FMT>) {
        const int odd = page & 1;
        const char* r0 = record(pp[0]);
        const char* r1 = record(pp[1]);
        if (r0 && r1) put_key_group<FMT>(r0, r1, kP * odd, kP * odd + kP, TileRows{rows.tile, rows.r0 - kP * odd, nullptr});
        else rows.clear(0, kP);
      }
    } else {
      const char* rec = record(pp[0]);
      const float one = 1.0f;   // FP8: codes, exact in f16; the attention kernel scales scores and outputs
      if (!rec) rows.clear(0, held);
      else if (values) put_values<FMT>(&one, rec, 0, held, rows);
      else if constexpr (kByte<FMT>) put_keys<FMT>(&one, rec, 0, held, rows);
    }
  }
  if (FMT != 8 && end > held) put_ring(ring, mod, tp, held, end, a.dtype, rows);
  rows.clear(end, kP);   // behind the last token: zeros, which a probability of zero leaves alone
  if (values) {
    bits = __reduce_or_sync(0xffffffffu, bits);
    if (lane == 0) reinterpret_cast<uint16_t*>(a.bad + 4 * at)[warp] = static_cast<uint16_t>(bits);
  }
}

template <int FMT>
cudaError_t run(const PromptArgs& a, cudaStream_t st) {
  void (*f)(PromptArgs) = tiles_kernel<FMT>;
  const cudaError_t c = prefer_max_shared(reinterpret_cast<const void*>(f));
  if (c != cudaSuccess) return c;
  return launch_behind(f, dim3(static_cast<unsigned>(a.kv_grid), static_cast<unsigned>(a.H), 2), dim3(kThreads), 0, st, a);
}

}  // namespace

cudaError_t launch_tiles(const PromptArgs& a, cudaStream_t st) {
  switch (a.bits) {
    case S4KV_BITS_INT8: return run<S4KV_BITS_INT8>(a, st);
    case 8: return run<8>(a, st);
    case 2: return run<2>(a, st);
    default: return run<4>(a, st);
  }
}

}  // namespace s4kv
