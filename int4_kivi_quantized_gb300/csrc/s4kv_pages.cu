// Page accounting on the device (s4kv_take_pages, s4kv_release_pages) and forks (s4kv_fork):
// refs[p] counts the block-table entries that name page p, 0 is free.
//
// Giving out pages is a scan: sequence i's pages are the free ones of rank need_1 + .. +
// need_(i-1) on, and the page of rank k is the k-th zero of refs. One CTA does it, as a scheduler's
// step asks for some hundred pages: it stops at the tile of refs where enough are found. What
// bounds it is latency: the launch, the lengths, one or two tiles, the entries. Measured under the profiler, cold
// caches: 32 sequences 9.4 us, 512 that take 1536 pages 11.9; with the release behind it, many in a captured
// graph, 8.4 and 10.9 (7.6 and 10.0 without a look at the entries first; entered by the thread that found a page
// 3.5 more for the 512). Bytes at the memory's rate would be 0.5.
//
// A fork then copies what both sequences would go on writing (the pages from the first
// unfinished one on, the rings), a CTA for each page, or head's rings, of each layer, 16 bytes a
// thread and load, eight loads in flight: bound by those bytes, read and written once. Measured: four
// forks of one 4-bit sequence of 1000 tokens, 4 layers, 8 heads: 10.3 us and 7.0; 64 forks of 16 prompts
// of 700 to 2048 10 us and 25.

#include "s4kv_pages.cuh"

namespace s4kv {
namespace {

constexpr int kThreads = 1024;
constexpr int kEach = 16;                     // neighbouring counts of a thread
constexpr int kTile = kThreads * kEach;
constexpr int kList = 4096;

__device__ __forceinline__ unsigned add_to(unsigned a, unsigned b) { return min(a + b, 0x7fffffffu); }   // (both below 2^31)

// Exclusive sum over the CTA, and the total, saturating.
__device__ __forceinline__ unsigned block_scan(unsigned x, unsigned& total) {
  __shared__ unsigned tot[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned s = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s = add_to(s, y);
  }
  __syncthreads();   // the totals of the call before are read
  if (lane == 31) tot[warp] = s;
  __syncthreads();
  unsigned t = tot[lane], before = 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned y = __shfl_up_sync(0xffffffffu, t, o);
    if (lane >= o) t = add_to(t, y);
  }
  total = __shfl_sync(0xffffffffu, t, 31);
  before = __shfl_sync(0xffffffffu, t, max(warp - 1, 0));
  const unsigned mine = __shfl_up_sync(0xffffffffu, s, 1);
  return add_to(warp > 0 ? before : 0u, lane > 0 ? mine : 0u);
}

__device__ __forceinline__ int pages_for(int tokens) { return static_cast<int>((static_cast<unsigned>(tokens) + kP - 1) / kP); }

// Sequence i of the call: its table row, and the entries [e0, e1) that it wants pages for.
struct Want {
  int row, e0, e1;
};
template <bool FORK>
__device__ __forceinline__ Want want_of(const PageArgs& a, int i) {
  if (FORK) {
    const int T = a.seq_lens[i];
    return Want{a.to[i], held_of(a.bits, T, a.R).done, pages_for(T)};
  }
  return Want{a.slot_ids ? a.slot_ids[i] : i, pages_for(a.from[i]), pages_for(a.to[i])};
}

template <bool FORK>
__global__ void __launch_bounds__(kThreads, 1) give_kernel(PageArgs a) {
  __shared__ unsigned pre[kMaxPageJobs + 1];                  // pages wanted by the sequences before
  __shared__ unsigned seen[kMaxPageRows / 32];                // rows, a bit each
  __shared__ unsigned list[kList];                            // two more such sets, then pages by rank
  __shared__ unsigned filled[FORK ? 1 : kMaxPageJobs / 32];   // sequences, a bit each: an entry to fill names a page
  unsigned* const twice = list;
  unsigned* const source = list + kMaxPageRows / 32;
  static_assert(kList >= 2 * (kMaxPageRows / 32), "both sets");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < (a.rows + 31) / 32; i += kThreads) {
    seen[i] = twice[i] = 0u;
    if (FORK) source[i] = 0u;
  }
  for (int i = tid; !FORK && i < (a.n + 31) / 32; i += kThreads) filled[i] = 0u;
  stream_wait();
  __syncthreads();
  auto row_ok = [&](int r) { return r >= 0 && r < a.rows; };
  auto bit = [&](const unsigned* set, int r) { return (set[r >> 5] >> (r & 31)) & 1u; };
  for (int i = tid; i < a.n; i += kThreads) {
    const int r = FORK ? a.to[i] : a.slot_ids ? a.slot_ids[i] : i;
    if (row_ok(r) && (atomicOr(&seen[r >> 5], 1u << (r & 31)) >> (r & 31)) & 1u) atomicOr(&twice[r >> 5], 1u << (r & 31));
    if (FORK && row_ok(a.from[i])) atomicOr(&source[a.from[i] >> 5], 1u << (a.from[i] & 31));
  }
  __syncthreads();
  // why sequence i gets nothing, whatever is free: 0 if it may
  auto refused = [&](int i, int& arg) -> int {
    const int r = FORK ? a.to[i] : a.slot_ids ? a.slot_ids[i] : i;
    arg = r;
    if (!row_ok(r) || bit(twice, r) || (FORK && (!row_ok(a.from[i]) || bit(source, r)))) return S4KV_DEV_BAD_SLOT;
    arg = i;
    if (FORK ? a.seq_lens[i] < 0 : (a.from[i] < 0 || a.to[i] < a.from[i])) return S4KV_DEV_BAD_LENGTH;
    if (pages_for(FORK ? a.seq_lens[i] : a.to[i]) > a.bt_stride) return S4KV_DEV_BAD_TABLE;
    return 0;
  };
  if (FORK) {   // a warp a fork: every layer and head of the source holds as many tokens, and what has to be copied is there
    for (int i = warp; i < a.n; i += kThreads / 32) {
      int arg, why = refused(i, arg);
      if (!why) {
        const int src = a.from[i], T = a.seq_lens[i], words = a.layers * a.H;
        const Held x = held_of(a.bits, T, a.R);
        auto page = [&](int e) { return e < x.held ? a.table[static_cast<long long>(src) * a.bt_stride + e] : 0; };
        auto length = [&](int k) { return k < words ? __ldcg(a.lens + (static_cast<size_t>(k / a.H) * a.max_slots + src) * a.H + k % a.H) : T; };
        auto outside = [&](int p) { return p < 0 || p >= a.num_pages; };
        const int p0 = page(x.done + lane), n0 = length(lane);   // (asked for together)
        bool hole = outside(p0), other = n0 != T;
        for (int e = x.done + 32 + lane; e < x.held; e += 32) hole = hole || outside(page(e));
        for (int k = 32 + lane; k < words; k += 32) other = other || length(k) != T;
        if (__any_sync(0xffffffffu, hole)) why = S4KV_DEV_BAD_PAGE;
        if (__any_sync(0xffffffffu, other)) why = S4KV_DEV_BAD_LENGTH;
      }
      if (lane == 0) {
        if (why) report(a.status, S4KV_ERR_DEVICE, why, arg);
        const Want w = want_of<FORK>(a, i);
        pre[i + 1] = why ? 0u : static_cast<unsigned>(w.e1 - w.e0);
        a.taken[i] = why ? -1 : 0;
      }
    }
  } else {
    for (int i = tid; i < a.n; i += kThreads) {
      int arg;
      const int why = refused(i, arg);
      if (why) report(a.status, S4KV_ERR_DEVICE, why, arg);
      const Want w = want_of<FORK>(a, i);
      pre[i + 1] = why ? 0u : static_cast<unsigned>(w.e1 - w.e0);
      a.taken[i] = why ? -1 : 0;
    }
  }
  __syncthreads();
  unsigned total;
  {   // sums in place: four neighbouring sequences a thread
    constexpr int kSeqs = kMaxPageJobs / kThreads;
    unsigned x[kSeqs], mine = 0;
#pragma unroll
    for (int k = 0; k < kSeqs; ++k) {
      x[k] = kSeqs * tid + k < a.n ? pre[kSeqs * tid + k + 1] : 0u;
      mine = add_to(mine, x[k]);
    }
    unsigned at = block_scan(mine, total);
#pragma unroll
    for (int k = 0; k < kSeqs; ++k) {
      at = add_to(at, x[k]);
      if (kSeqs * tid + k < a.n) pre[kSeqs * tid + k + 1] = at;
    }
    if (tid == 0) pre[0] = 0u;
  }
  // free pages of a tile of counts: a bit for each of this thread's
  auto look = [&](int base) -> unsigned {
    unsigned z = 0;
    const int p = base + tid * kEach;
    if (p + kEach <= a.num_pages) {
#pragma unroll
      for (int k = 0; k < kEach / 4; ++k) {
        const int4 v = *reinterpret_cast<const int4*>(a.refs + p + 4 * k);
        z |= ((v.x == 0 ? 1u : 0u) | (v.y == 0 ? 2u : 0u) | (v.z == 0 ? 4u : 0u) | (v.w == 0 ? 8u : 0u)) << (4 * k);
      }
    } else {
      for (int k = 0; k < kEach; ++k)
        if (p + k < a.num_pages && a.refs[p + k] == 0) z |= 1u << k;
    }
    return z;
  };
  auto owner_of = [&](unsigned k) -> int {   // of the page of rank k: the last sequence with pre <= k
    int lo = 0, hi = a.n - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pre[mid] <= k) lo = mid; else hi = mid - 1;
    }
    return lo;
  };
  // The entries for the pages of ranks r + tid, r + tid + kThreads, ..: whose, and where (row -1: none).
  constexpr int kMine = kList / kThreads;
  auto entries_of = [&](unsigned r, unsigned end, Want (&w)[kMine], int (&who)[kMine]) {
#pragma unroll
    for (int c = 0; c < kMine; ++c) {
      const unsigned k = r + tid + c * kThreads;
      w[c].row = -1;
      if (k >= end) continue;
      who[c] = owner_of(k);
      w[c] = want_of<FORK>(a, who[c]);
      w[c].e0 += k - pre[who[c]];
    }
  };
  auto entry = [&](const Want& w) -> int& { return a.table[static_cast<long long>(w.row) * a.bt_stride + w.e0]; };
  __syncthreads();   // the sums are there
  const unsigned most = min(total, static_cast<unsigned>(a.num_pages));   // ranks that there may be
  Want first_w[kMine];
  int first_who[kMine];
  entries_of(0, most, first_w, first_who);
  unsigned z0 = 0;
  if (!FORK) {   // entries that name a page (a fork's new row is overwritten)
    int old[kMine];
#pragma unroll
    for (int c = 0; c < kMine; ++c) old[c] = first_w[c].row >= 0 ? entry(first_w[c]) : -1;
    if (total > 0) z0 = look(0);
#pragma unroll
    for (int c = 0; c < kMine; ++c)
      if (old[c] != -1) atomicOr(&filled[first_who[c] >> 5], 1u << (first_who[c] & 31));
    for (unsigned r = kList; r < most; r += kList) {
      Want w[kMine];
      int who[kMine];
      entries_of(r, most, w, who);
#pragma unroll
      for (int c = 0; c < kMine; ++c) old[c] = w[c].row >= 0 ? entry(w[c]) : -1;
#pragma unroll
      for (int c = 0; c < kMine; ++c)
        if (old[c] != -1) atomicOr(&filled[who[c] >> 5], 1u << (who[c] & 31));
    }
  } else if (total > 0) {
    z0 = look(0);
  }
  // enough of them, or all there are (the last tile looked at is at hand again if it is the first)
  unsigned found = 0;
  for (int base = 0; found < total && base < a.num_pages; base += kTile) {
    const unsigned z = base == 0 ? z0 : look(base);
    unsigned here;
    block_scan(__popc(z), here);
    found = add_to(found, here);
  }
  __syncthreads();
  unsigned granted = total;
  if (found < total) {   // sequences in order, while they can be served
    int lo = 0, hi = a.n;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pre[mid] <= found) lo = mid; else hi = mid - 1;
    }
    granted = pre[lo];
  }
  for (int i = tid; i < a.n; i += kThreads) {
    const Want w = want_of<FORK>(a, i);
    if (a.taken[i] != 0 || w.e1 <= w.e0) continue;
    const bool room = pre[i + 1] <= granted, full = !FORK && bit(filled, i);
    if (room && full) report(a.status, S4KV_ERR_DEVICE, S4KV_DEV_BAD_TABLE, i);
    a.taken[i] = room && !full ? w.e1 - w.e0 : -1;
  }
  unsigned rank0 = 0;
  for (int base = 0; rank0 < granted && base < a.num_pages; base += kTile) {
    unsigned z = base == 0 ? z0 : look(base), here;
    const unsigned k0 = rank0 + block_scan(__popc(z), here), end = min(rank0 + here, granted);
    // through a list by rank, so that the pages of one thread's counts are every thread's to enter
    for (unsigned r = rank0; r < end; r += kList) {
      __syncthreads();
      unsigned k = k0;
      for (unsigned y = z; y && k < end; y &= y - 1, ++k)
        if (k - r < kList) list[k - r] = base + tid * kEach + __ffs(y) - 1;
      __syncthreads();
      Want w[kMine];
      int who[kMine];
      if (r == 0) {
#pragma unroll
        for (int c = 0; c < kMine; ++c) {
          w[c] = first_w[c];
          who[c] = first_who[c];
        }
      } else {
        entries_of(r, end, w, who);
      }
#pragma unroll
      for (int c = 0; c < kMine; ++c) {
        k = r + tid + c * kThreads;
        if (k >= end || (!FORK && bit(filled, who[c]))) continue;   // (filled: its pages stay free)
        const int p = list[k - r];
        entry(w[c]) = p;
        a.refs[p] = 1;
      }
    }
    rank0 += here;
  }
}

constexpr int kRelease = 256;
__global__ void __launch_bounds__(kRelease) release_kernel(PageArgs a) {
  stream_wait();
  const int i = blockIdx.x, row = a.slot_ids ? a.slot_ids[i] : i, first = a.from[i], last = a.to[i];
  int why = 0;
  if (row < 0 || row >= a.rows) why = S4KV_DEV_BAD_SLOT;
  else if (first < 0 || last < 0) why = S4KV_DEV_BAD_LENGTH;
  else if (last > first && pages_for(last) > a.bt_stride) why = S4KV_DEV_BAD_TABLE;
  if (why) {
    if (threadIdx.x == 0 && blockIdx.y == 0) report(a.status, S4KV_ERR_DEVICE, why, why == S4KV_DEV_BAD_SLOT ? row : i);
    return;
  }
  const int e1 = last > first ? pages_for(last) : 0;
  int* entries = a.table + static_cast<long long>(row) * a.bt_stride;
  for (int e = pages_for(first) + blockIdx.y * kRelease + threadIdx.x; e < e1; e += gridDim.y * kRelease) {
    const int p = atomicExch(entries + e, -1);   // (a row named twice: only one of them gets it)
    if (p == -1) continue;
    if (p < 0 || p >= a.num_pages) {
      report(a.status, S4KV_ERR_DEVICE, S4KV_DEV_BAD_PAGE, p);
    } else if (atomicSub(a.refs + p, 1) <= 0) {   // nobody had it
      atomicAdd(a.refs + p, 1);
      report(a.status, S4KV_ERR_DEVICE, S4KV_DEV_BAD_PAGE, p);
    }
  }
}

constexpr int kCopy = 256;
// `bytes` (a multiple of 16) by the CTA.
__device__ __forceinline__ void copy_bytes(char* dst, const char* src, int bytes) {
  const int n = bytes / 16;
  uint4* d = reinterpret_cast<uint4*>(dst);
  const uint4* s = reinterpret_cast<const uint4*>(src);
  constexpr int kAhead = 8;
  for (int i0 = threadIdx.x; i0 < n; i0 += kAhead * kCopy) {
    uint4 v[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (i0 + k * kCopy < n) v[k] = s[i0 + k * kCopy];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (i0 + k * kCopy < n) d[i0 + k * kCopy] = v[k];
  }
}

// blockIdx: x the part (page, head's rings and length, the shared entries), y the layer, z the fork.
__global__ void __launch_bounds__(kCopy) fork_kernel(PageArgs a) {
  stream_wait();
  const int i = blockIdx.z, layer = blockIdx.y, part = blockIdx.x;
  if (a.taken[i] < 0) return;
  const int src = a.from[i], dst = a.to[i], T = a.seq_lens[i];
  const Held x = held_of(a.bits, T, a.R);
  const int* from = a.table + static_cast<long long>(src) * a.bt_stride;
  int* to = a.table + static_cast<long long>(dst) * a.bt_stride;
  char* base = a.pool_layers + layer * a.layer_stride;
  if (part < a.pages_at_most) {
    const int e = x.done + part;
    if (e >= x.held) return;
    const int p = from[e], q = to[e];
    if (p < 0 || p >= a.num_pages) return;   // (not so when the launch before this one looked: the table may not change meanwhile)
    copy_bytes(base + q * a.page_bytes, base + p * a.page_bytes, static_cast<int>(a.page_bytes));
  } else if (part < a.pages_at_most + a.H) {
    const int h = part - a.pages_at_most;
    char* k = base + a.kring_offset + h * a.kring_head;
    char* v = base + a.vring_offset + h * a.vring_head;
    copy_bytes(k + dst * a.kring_slot, k + src * a.kring_slot, x.krows * kD * 2);
    copy_bytes(v + dst * a.vring_slot, v + src * a.vring_slot, x.vrows * kD * 2);
    if (threadIdx.x == 0) a.lens[(static_cast<size_t>(layer) * a.max_slots + dst) * a.H + h] = T;
  } else if (layer == 0) {
    for (int e = (part - a.pages_at_most - a.H) * kCopy + threadIdx.x; e < x.done; e += kCopy * (gridDim.x - a.pages_at_most - a.H)) {
      int p = from[e];
      if (p < -1 || p >= a.num_pages) {
        report(a.status, S4KV_ERR_DEVICE, S4KV_DEV_BAD_PAGE, p);
        p = -1;
      }
      to[e] = p;
      if (p >= 0) atomicAdd(a.refs + p, 1);   // (-1: given away already)
    }
  }
}

}  // namespace

cudaError_t launch_take(const PageArgs& a, cudaStream_t st) {
  return launch_behind(give_kernel<false>, dim3(1), dim3(kThreads), 0, st, a);
}

cudaError_t launch_release(const PageArgs& a, cudaStream_t st) {
  int more = (a.bt_stride + kRelease - 1) / kRelease;   // CTAs of a long row
  if (more > 16) more = 16;
  return launch_behind(release_kernel, dim3(static_cast<unsigned>(a.n), static_cast<unsigned>(more)), dim3(kRelease), 0, st, a);
}

cudaError_t launch_fork(const PageArgs& a, cudaStream_t st) {
  cudaError_t e = launch_behind(give_kernel<true>, dim3(1), dim3(kThreads), 0, st, a);
  if (e != cudaSuccess) return e;
  const unsigned parts = static_cast<unsigned>(a.pages_at_most + a.H);
  // the shared entries: with the first layer's parts (y = 0), a CTA for every 256
  int more = (a.bt_stride + kCopy - 1) / kCopy;
  if (more > 8) more = 8;
  return launch_behind(fork_kernel, dim3(parts + more, static_cast<unsigned>(a.layers), static_cast<unsigned>(a.n)), dim3(kCopy), 0, st, a);
}

}  // namespace s4kv
