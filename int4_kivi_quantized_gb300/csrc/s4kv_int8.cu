// Write side of INT8 block pages: s4kv_append and s4kv_append_rope on a cache
// whose pages hold 8-bit integers with one scale per 16-token block, kv head and
// tensor (the format and the quantizer are in include/s4kv.h).
//
// A block's codes need its largest magnitude, so a block is quantized when its
// 16 tokens are there: once, from 16-bit rows, whatever the chunks they came in.
// The tokens of an unfinished block wait in rings.
//
// Work items, one warp each:
//  * a block made only of new tokens: both tensors of one kv head, 8 KiB of rows
//    in flight per warp, reduced, coded and written as a record in place;
//  * the edge of a (sequence, head): the block that ring rows and new rows
//    complete together, then the rows left over into the rings (one warp, so ring
//    rows are read before they are overwritten), and the stored length;
//  * with a rotation, 16 heads of one query row.
// This unit is compiled without FMA contraction; every rounding is spelled out.

#include "s4kv_common.cuh"
#include "s4kv_rope.cuh"

namespace s4kv {
namespace {

using R8 = Rec<S4KV_BITS_INT8>;
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
#ifndef S4KV_INT8_CTAS
#define S4KV_INT8_CTAS 4
#endif
// Resident CTAs per SM the registers are budgeted for: a rotation holds 32 angles
// beside the block's 64 words.
template <bool ROPE> constexpr int kCtas = ROPE ? 3 : S4KV_INT8_CTAS;
constexpr float kTiny = 7.8886091e-31f;   // 2^-100
// 1.5 * 2^23 + 128: t + kMagic has round_half_even(t) + 128 in its low byte
constexpr float kMagic = 12583040.0f;

// Largest |x| bit pattern of two packed 16-bit pairs (NaN patterns are the largest).
__device__ __forceinline__ uint32_t absmax2(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7fff7fffu); }
__device__ __forceinline__ uint32_t absmax8(uint32_t m, uint4 w) {
  return absmax2(absmax2(absmax2(absmax2(m, w.x), w.y), w.z), w.w);
}

struct Scale {
  float s, inv;
};
template <int DT>
__device__ __forceinline__ Scale scale_of(uint32_t m) {
  const unsigned top = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
  const float A = widen16(static_cast<uint16_t>(top), DT);
  Scale r;
  r.s = A < kTiny ? 0.0f : __fdiv_rn(A, 127.0f);
  r.inv = A < kTiny ? 0.0f : __fdiv_rn(127.0f, A);
  return r;
}

template <int DT>
__device__ __forceinline__ uint32_t coded(uint32_t half16, float inv) {   // low byte: code + 128
  return __float_as_uint(__fadd_rn(__fmul_rn(widen16(static_cast<uint16_t>(half16), DT), inv), kMagic));
}
__device__ __forceinline__ uint32_t bytes4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}
__device__ __forceinline__ uint32_t word(const uint4& w, int i) { return i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w; }

struct Seq {
  int i, slot, T0, T1, c0;
  bool ok;
};

// Sequence i's row range, lengths and slot, checked; errors are reported by
// `tell` warps only (one per sequence), all of a sequence's items agree on them.
template <bool ROPE>
__device__ __forceinline__ Seq sequence(const AppendArgs& a, int i, int h, bool tell) {
  Seq s;
  s.i = i;
  s.slot = a.slot_ids ? a.slot_ids[i] : i;
  const int len = a.seq_lens_before[i];
  if (a.step) {
    s.c0 = i;
    s.T1 = len;
    s.T0 = len - 1;
  } else {
    s.c0 = a.cu_new[i];
    s.T0 = len;
    s.T1 = len + a.cu_new[i + 1] - s.c0;
  }
  int bad = 0, arg = i;
  if (s.slot < 0 || s.slot >= a.max_slots) {
    bad = S4KV_DEV_BAD_SLOT;
    arg = s.slot;
  } else if (s.T0 < 0 || (a.step && s.T1 > a.max_len)) {
    bad = S4KV_DEV_BAD_LENGTH;
  } else if (static_cast<long long>(a.bt_stride) * kP < s.T1) {
    bad = S4KV_DEV_BAD_TABLE;
  } else if (ROPE && s.T1 > a.rope.max_pos) {
    bad = S4KV_DEV_BAD_POSITION;
  } else if (s.T0 != 0) {
    // the length this append starts from, or the one its edge item may have stored already
    const int stored = __ldcg(a.lens + s.slot * a.H + h);
    if (stored != s.T0 && stored != s.T1) bad = S4KV_DEV_BAD_LENGTH;
    if (tell && stored != s.T0) bad = S4KV_DEV_BAD_LENGTH;   // (the edge item is the only writer)
  }
  s.ok = bad == 0;
  if (bad && tell && (threadIdx.x & 31) == 0) report(a.status, S4KV_ERR_DEVICE, bad, arg);
  return s;
}

__device__ __forceinline__ char* record(const AppendArgs& a, const Seq& s, int page, int h) {
  const int pp = a.block_table[static_cast<long long>(s.i) * a.bt_stride + page];
  if (pp < 0 || pp >= a.num_pages) {
    if ((threadIdx.x & 31) == 0) report(a.status, S4KV_ERR_DEVICE, S4KV_DEV_BAD_PAGE, pp);
    return nullptr;
  }
  return a.pages + (static_cast<long long>(pp) * a.H + h) * R8::kBytes;
}

// One whole block into its record. Token t0 + x comes from ring row x for x <
// ring_rows (its key already turned), else from the input.
//
// Keys: lane l holds tokens 4r + l / 8 (r = 0..3), chunks l % 8 and l % 8 + 8 of
// 8 channels: the operands of the record's 16-byte key words, and with a full
// rotation both members of every pair. Values: lane (a, b) = (l / 4, l % 4) holds
// tokens 2b, 2b+1, 2b+8, 2b+9 and chunks a and a + 8, which make its value words.
// Both loads read whole 128-byte lines.
template <int DT, bool ROPE>
__device__ __forceinline__ void whole_block(const AppendArgs& a, const Seq& s, int h, int page, int ring_rows) {
  const int lane = threadIdx.x & 31, t0 = page * kP;
  const uint16_t* kin = a.k + (static_cast<long long>(s.c0 + t0 - s.T0) * a.H + h) * kD;   // row of token t0 (may lie before the input when ring rows come first)
  const uint16_t* vin = a.v + (static_cast<long long>(s.c0 + t0 - s.T0) * a.H + h) * kD;
  const uint16_t* kring = reinterpret_cast<const uint16_t*>(a.kring) + s.slot * a.kring_slot + h * a.kring_head;
  const uint16_t* vring = reinterpret_cast<const uint16_t*>(a.vring) + s.slot * a.vring_slot + h * a.vring_head;
  const long long step = static_cast<long long>(a.H) * kD;
  uint4 k[8], v[8];
  const int kc = lane & 7, kr = lane >> 3;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int x = 4 * r + kr;
    const uint4* row = reinterpret_cast<const uint4*>(x < ring_rows ? kring + x * kD : kin + x * step);
    k[2 * r] = row[kc];
    k[2 * r + 1] = row[kc + 8];
  }
  const int ca = lane >> 2, tb = lane & 3;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int x = 2 * tb + (j & 1) + 8 * (j >> 1);
    const uint4* row = reinterpret_cast<const uint4*>(x < ring_rows ? vring + x * kD : vin + x * step);
    v[2 * j] = row[ca];
    v[2 * j + 1] = row[ca + 8];
  }
  char* rec = record(a, s, page, h);
  if constexpr (ROPE) {
    if (a.rope.interleaved || a.rope.dim == kD) {
      // a lane's chunks c and c + 8 are a unit of the rotation; the next row's angles
      // load while this one turns
      rope::Unit u[2];
      rope::unit_chunks(a.rope, kc, u[0]);
      u[1] = u[0];
      rope::unit_angles(a.rope, t0 + kr, u[0]);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (r < 3) rope::unit_angles(a.rope, t0 + 4 * (r + 1) + kr, u[(r + 1) & 1]);
        if (4 * r + kr >= ring_rows) rope::turn_unit<DT>(a.rope, u[r & 1], k[2 * r], k[2 * r + 1]);
      }
    } else {   // a pair's other chunk is another lane's
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int x = 4 * r + kr;
        if (x >= ring_rows) {
          const uint4* row = reinterpret_cast<const uint4*>(kin + x * step);
          const uint4 plo = row[rope::partner(a.rope, kc)], phi = row[rope::partner(a.rope, kc + 8)];
          k[2 * r] = rope::turn(a.rope, t0 + x, kc, k[2 * r], plo, DT);
          k[2 * r + 1] = rope::turn(a.rope, t0 + x, kc + 8, k[2 * r + 1], phi, DT);
        }
      }
    }
  }
  uint32_t mk = 0, mv = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    mk = absmax8(mk, k[i]);
    mv = absmax8(mv, v[i]);
  }
  const Scale ks = scale_of<DT>(mk), vs = scale_of<DT>(mv);
  if (!rec) return;
#pragma unroll
  for (int r = 0; r < 2; ++r) {   // tokens ta = 4r + l / 8 and ta + 8
    const int ta = 4 * r + kr;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const uint4 x = k[2 * r + half], y = k[2 * (r + 2) + half];
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t p = word(x, i), q = word(y, i);
        w[i] = bytes4(coded<DT>(p & 0xffffu, ks.inv), coded<DT>(p >> 16, ks.inv), coded<DT>(q & 0xffffu, ks.inv),
                      coded<DT>(q >> 16, ks.inv));
      }
      const int c = kc + 8 * half;   // channels 8c .. 8c+7: word kp = c % 4 of lane 4 ta + c / 4
      *reinterpret_cast<uint4*>(rec + R8::kKc + (c & 3) * 512 + (4 * ta + (c >> 2)) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
#pragma unroll
  for (int kp = 0; kp < 4; ++kp) {   // channels 8 ca + m and 64 + 8 ca + m, m = 2 kp, 2 kp + 1
    uint32_t w[4];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int j = 0; j < 2; ++j) {   // tokens 2b, 2b + 1 | 2b + 8, 2b + 9
        const uint32_t l0 = word(v[4 * j], kp), l1 = word(v[4 * j + 2], kp);
        const uint32_t h0 = word(v[4 * j + 1], kp), h1 = word(v[4 * j + 3], kp);
        const int sh = 16 * u;
        w[2 * u + j] = bytes4(coded<DT>((l0 >> sh) & 0xffffu, vs.inv), coded<DT>((l1 >> sh) & 0xffffu, vs.inv),
                              coded<DT>((h0 >> sh) & 0xffffu, vs.inv), coded<DT>((h1 >> sh) & 0xffffu, vs.inv));
      }
    *reinterpret_cast<uint4*>(rec + R8::kVc + kp * 512 + lane * 16) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  if (lane == 0) *reinterpret_cast<float2*>(rec + R8::kKs) = make_float2(ks.s, vs.s);
}

// The edge of (sequence, head): see the top of the file.
template <int DT, bool ROPE>
__device__ __forceinline__ void edge(const AppendArgs& a, int i, int h) {
  const int lane = threadIdx.x & 31;
  const Seq s = sequence<ROPE>(a, i, h, true);
  if (!s.ok) return;
  const int head = s.T0 % kP;
  if (head != 0 && s.T0 - head + kP <= s.T1) {
    whole_block<DT, ROPE>(a, s, h, s.T0 / kP, head);
    __syncwarp();   // every lane has read its ring rows
  }
  // tokens [max(T0, last block), T1) wait in the rings
  const int from = max(s.T0, s.T1 - s.T1 % kP), n = s.T1 - from;
  const long long in = (static_cast<long long>(s.c0 + from - s.T0) * a.H + h) * kD;
  uint16_t* kring = reinterpret_cast<uint16_t*>(a.kring) + s.slot * a.kring_slot + h * a.kring_head;
  uint16_t* vring = reinterpret_cast<uint16_t*>(a.vring) + s.slot * a.vring_slot + h * a.vring_head;
  for (int q = lane; q < 16 * n; q += 32) {
    const int t = from + (q >> 4), c = q & 15;
    const long long off = in + static_cast<long long>(q >> 4) * a.H * kD;
    uint4 x;
    if constexpr (ROPE) x = rope::turned_chunk(a.rope, a.k + off, t, c, DT);
    else x = reinterpret_cast<const uint4*>(a.k + off)[c];
    const uint4 y = reinterpret_cast<const uint4*>(a.v + off)[c];
    reinterpret_cast<uint4*>(kring + (t % kP) * kD)[c] = x;
    reinterpret_cast<uint4*>(vring + (t % kP) * kD)[c] = y;
  }
  if (lane == 0) __stcg(a.lens + s.slot * a.H + h, s.T1);
}

template <int DT, bool ROPE>
__global__ void __launch_bounds__(kThreads, kCtas<ROPE>) append_int8_kernel(AppendArgs a) {
  if (!a.step) {   // a malformed call (see s4kv_append): nothing is read or written
    int bad = a.cu_new[0] != 0 || a.cu_new[a.n] != a.num_new;
    for (int i = threadIdx.x; i < a.n; i += kThreads) {
      const int ni = a.cu_new[i + 1] - a.cu_new[i], T0 = a.seq_lens_before[i];
      bad |= ni < 0 || ni > (1 << 30) || T0 < 0 || T0 > (1 << 30);
    }
    bad = __syncthreads_or(bad);
    if (bad) {
      if (blockIdx.x == 0 && threadIdx.x == 0) report(a.status, S4KV_ERR_DEVICE, S4KV_DEV_BAD_CU, a.n);
      return;
    }
  }
  // Block slots: the whole new block whose first input row is x has slot
  // ceil(x / 16). Blocks of a sequence are 16 rows apart and the next sequence
  // starts past the last one's 16 rows, so slots are distinct, and row 16 slot
  // lies inside the block: it names the sequence.
  const int slots = a.step ? 0 : (a.num_new + kP - 1) / kP;
  const long long blocks = static_cast<long long>(slots) * a.H;
  const long long edges = blocks + static_cast<long long>(a.n) * a.H;
  const long long total = edges + (ROPE ? rope::query_items(a.rope, a.num_new) : 0);
  for (long long it = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5); it < total;
       it += static_cast<long long>(gridDim.x) * kWarps) {
    if (it < blocks) {
      const int slot = static_cast<int>(it / a.H), h = static_cast<int>(it - static_cast<long long>(slot) * a.H);
      const int row = slot * kP;
      const int i = rope::sequence_of_row(a.cu_new, a.n, row);
      const int page = (a.seq_lens_before[i] + row - a.cu_new[i]) / kP;
      const Seq s = sequence<ROPE>(a, i, h, false);
      if (s.ok && page * kP >= s.T0 && page * kP + kP <= s.T1) whole_block<DT, ROPE>(a, s, h, page, 0);
    } else if (it < edges) {
      const long long e = it - blocks;
      edge<DT, ROPE>(a, static_cast<int>(e / a.H), static_cast<int>(e % a.H));
    } else if constexpr (ROPE) {
      rope::query_item<DT>(a, it - edges);
    }
    __syncwarp();
  }
}

}  // namespace

cudaError_t launch_append_int8(const AppendArgs& a, int num_sms, cudaStream_t st) {
  const bool turn = a.rope.table != nullptr;
  void (*kern)(AppendArgs);
  if (a.dtype == S4KV_BF16) kern = turn ? append_int8_kernel<S4KV_BF16, true> : append_int8_kernel<S4KV_BF16, false>;
  else kern = turn ? append_int8_kernel<S4KV_F16, true> : append_int8_kernel<S4KV_F16, false>;
  const cudaError_t c = prefer_max_shared(reinterpret_cast<const void*>(kern));
  if (c != cudaSuccess) return c;
  const long long slots = a.step ? 0 : (a.num_new + kP - 1) / kP;
  const long long items = (slots + a.n) * a.H + rope::query_items(a.rope, a.num_new);
  const long long want = (items + kWarps - 1) / kWarps, cap = static_cast<long long>(num_sms) * (turn ? kCtas<true> : kCtas<false>);
  kern<<<static_cast<unsigned>(want < cap ? want : cap), kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace s4kv
