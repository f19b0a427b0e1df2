// Write side of the 8-bit pages: s4kv_append and s4kv_append_rope on INT8 block
// pages, and s4kv_append_rope on FP8 pages (formats and quantizers in
// include/s4kv.h).
//
// An INT8 block's codes need its largest magnitude, so a block is quantized when its
// 16 tokens are there: once, from 16-bit rows, whatever the chunks they came in.
// The tokens of an unfinished block wait in rings. FP8 tokens go to their page on
// arrival.
//
// Work items, one warp each:
//  * a page made only of new tokens: both tensors of one kv head. A warp's next page
//    loads (cp.async, each lane the 16-byte pieces that it will need itself, so no
//    barrier) while this one is reduced, coded and written as a whole record;
//  * the edge of a (sequence, head), keys and values by two warps of a CTA: the page
//    that earlier and new tokens share, the last page if it is not full, and the
//    stored length;
//  * with a rotation, 16 heads of one query row, in CTAs of their own.
// 512 bytes of rows in and 258 (256) of record out per token and kv head: bound by
// those bytes, with the arithmetic of a rotation and a code per element close behind.
// Measured (16000 tokens, 8 kv heads, bf16; bytes at a plain copy's 6783 GB/s): INT8
// 16.4 us (bytes 14.3), rotated 23.7, with 32 query heads 67 (52.5); FP8 rotated 25 and 68.
// INT8, behind 1000 stored tokens of each of 8 sequences, whose lengths every item looks at:
// 19.5. One token of each of 128 sequences with its rotation and query: 5.
// This unit is compiled without FMA contraction; every rounding is spelled out.

#include "s4kv_common.cuh"
#include "s4kv_rope.cuh"

#include <cuda_fp8.h>

namespace s4kv {
namespace {

constexpr int kI8 = S4KV_BITS_INT8;
using R8 = Rec<kI8>;
static_assert(R8::kKc == Rec<8>::kKc && R8::kVc == Rec<8>::kVc, "both formats keep keys, then values");
constexpr int kWarps = 4;
static_assert(kWarps == 4, "two pairs of warps, a barrier each");
constexpr int kThreads = 32 * kWarps;
// (plain appends of 16000 tokens at 3 / 4 / 5: 17.4 / 16.4 / 15.9 us; rotated with 32 query
// heads 71 / 67 / 76)
#ifndef S4KV_APPEND8_CTAS
#define S4KV_APPEND8_CTAS 4
#endif
constexpr int kCtas = S4KV_APPEND8_CTAS;   // resident CTAs per SM the registers are budgeted for
// Query items (16 heads of a row) that turn in the time of a page. CTAs of their own, so
// that both go on side by side: 16000 tokens, 8 kv heads, 32 query heads 67 us (bytes:
// 52.5), against 73 where each warp does pages, then queries; with 1 / 2 / 3 here 79 /
// 67 / 71.
constexpr long long kPageQueries = 2;
constexpr int kStage = 16 * 512;           // a warp's page in flight: keys, then values
constexpr float kTiny = 7.8886091e-31f;    // 2^-100
// 1.5 * 2^23 + 128: t + kMagic has round_half_even(t) + 128 in its low byte
constexpr float kMagic = 12583040.0f;

// Largest |x| bit pattern of two packed 16-bit pairs (NaN patterns are the largest).
__device__ __forceinline__ uint32_t absmax2(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7fff7fffu); }
__device__ __forceinline__ uint32_t absmax8(uint32_t m, uint4 w) {
  return absmax2(absmax2(absmax2(absmax2(m, w.x), w.y), w.z), w.w);
}

// How a block's elements become bytes: INT8 by its own scale, FP8 by the head's.
struct Coder {
  float s;     // scale: INT8 A / 127; FP8 the head's
  float inv;   // INT8 127 / A; FP8 (MUL) 1 / s
};
// FP8 codes are those of x / s; where s is a power of two x (1 / s) is the same number.
__device__ __forceinline__ bool power_of_two(float s) {
  const uint32_t b = __float_as_uint(s);
  return (b & 0x7fffffu) == 0 && b >= 0x01000000u && b < 0x7e000000u;   // 1 / s is normal too
}
template <int FMT, int DT>
__device__ __forceinline__ Coder coder(const uint4 (&x)[8], float head_scale) {
  Coder c;
  if constexpr (FMT == kI8) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = absmax8(m, x[i]);
    const unsigned top = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
    const float A = widen16(static_cast<uint16_t>(top), DT);
    c.s = A < kTiny ? 0.0f : __fdiv_rn(A, 127.0f);
    c.inv = A < kTiny ? 0.0f : __fdiv_rn(127.0f, A);
  } else {
    c.s = head_scale;
    c.inv = __frcp_rn(head_scale);
  }
  return c;
}

// Codes of a packed pair (low element first) in the low 16 bits. MUL (FP8): by the
// inverse instead of the quotient.
template <int FMT, int DT, bool MUL>
__device__ __forceinline__ uint32_t code_pair(uint32_t w, const Coder& c) {
  const float x = widen16(static_cast<uint16_t>(w & 0xffff), DT), y = widen16(static_cast<uint16_t>(w >> 16), DT);
  if constexpr (FMT == kI8) {
    return __byte_perm(__float_as_uint(__fadd_rn(__fmul_rn(x, c.inv), kMagic)),
                       __float_as_uint(__fadd_rn(__fmul_rn(y, c.inv), kMagic)), 0x0040);
  } else {
    const float2 q = MUL ? make_float2(__fmul_rn(x, c.inv), __fmul_rn(y, c.inv))
                         : make_float2(__fdiv_rn(x, c.s), __fdiv_rn(y, c.s));
    return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3)) & 0xffffu;
  }
}

__device__ __forceinline__ uint32_t word(const uint4& w, int i) { return i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w; }
__device__ __forceinline__ uint4 blend(uint4 fresh, uint4 old, uint32_t k0, uint32_t k1, uint32_t k2, uint32_t k3) {
  return make_uint4((fresh.x & k0) | (old.x & ~k0), (fresh.y & k1) | (old.y & ~k1), (fresh.z & k2) | (old.z & ~k2),
                    (fresh.w & k3) | (old.w & ~k3));
}

// Keys of a block: lane l holds tokens 4r + l / 8 (r = 0..3) in k[2r] (chunk l % 8 of
// 8 channels) and k[2r + 1] (chunk l % 8 + 8), which make whole 16-byte key words,
// and with a full rotation both members of every pair. keep: the page's tokens
// below it stay as they are (FP8).
template <int FMT, int DT, bool MUL>
__device__ __forceinline__ void put_keys_by(char* rec, const uint4 (&k)[8], const Coder& cd, int keep) {
  const int lane = threadIdx.x & 31, kc = lane & 7, kr = lane >> 3;
#pragma unroll
  for (int r = 0; r < 2; ++r) {   // tokens ta and ta + 8
    const int ta = 4 * r + kr;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const uint4 x = k[2 * r + half], y = k[2 * (r + 2) + half];
      uint4 w;
      w.x = __byte_perm(code_pair<FMT, DT, MUL>(x.x, cd), code_pair<FMT, DT, MUL>(y.x, cd), 0x5410);
      w.y = __byte_perm(code_pair<FMT, DT, MUL>(x.y, cd), code_pair<FMT, DT, MUL>(y.y, cd), 0x5410);
      w.z = __byte_perm(code_pair<FMT, DT, MUL>(x.z, cd), code_pair<FMT, DT, MUL>(y.z, cd), 0x5410);
      w.w = __byte_perm(code_pair<FMT, DT, MUL>(x.w, cd), code_pair<FMT, DT, MUL>(y.w, cd), 0x5410);
      const int c = kc + 8 * half;   // channels 8c .. 8c+7: word c % 4 of lane 4 ta + c / 4
      uint4* dst = reinterpret_cast<uint4*>(rec + R8::kKc + (c & 3) * 512 + (4 * ta + (c >> 2)) * 16);
      if (FMT == 8 && keep > 0) {
        const uint32_t m = (ta >= keep ? 0x0000ffffu : 0u) | (ta + 8 >= keep ? 0xffff0000u : 0u);
        w = blend(w, *dst, m, m, m, m);
      }
      *dst = w;
    }
  }
}

// Values: lane (a, b) = (l / 4, l % 4) holds tokens 2b, 2b+1, 2b+8, 2b+9 (j = 0..3)
// in v[2j] (chunk a) and v[2j + 1] (chunk a + 8).
template <int FMT, int DT, bool MUL>
__device__ __forceinline__ void put_values_by(char* rec, const uint4 (&v)[8], const Coder& cd, int keep) {
  const int lane = threadIdx.x & 31;
  // t[half][m]: channel m of chunk a + 8 half as bytes of the four tokens
  uint32_t t[2][8];
#pragma unroll
  for (int half = 0; half < 2; ++half)
#pragma unroll
    for (int i = 0; i < 4; ++i) {   // channels 2i, 2i + 1
      const uint32_t p0 = code_pair<FMT, DT, MUL>(word(v[half], i), cd), p1 = code_pair<FMT, DT, MUL>(word(v[2 + half], i), cd);
      const uint32_t p2 = code_pair<FMT, DT, MUL>(word(v[4 + half], i), cd), p3 = code_pair<FMT, DT, MUL>(word(v[6 + half], i), cd);
      const uint32_t lo = __byte_perm(p0, p1, 0x5140), hi = __byte_perm(p2, p3, 0x5140);   // (c0t0, c0t1, c1t0, c1t1)
      t[half][2 * i] = __byte_perm(lo, hi, 0x5410);
      t[half][2 * i + 1] = __byte_perm(lo, hi, 0x7632);
    }
  if constexpr (FMT == 8) {
    // an FP8 value word holds channel a of every chunk: an 8 x 8 transpose over the
    // lanes of one b (bits 2..4 of the lane), exchanging half of the entries a step
#pragma unroll
    for (int s = 1; s < 8; s <<= 1) {
      const bool up = (lane >> 2) & s;
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int m = 0; m < 8; ++m)
          if (!(m & s)) {
            const uint32_t send = up ? t[half][m] : t[half][m | s];
            const uint32_t got = __shfl_xor_sync(0xffffffffu, send, s << 2);
            if (up) t[half][m] = got; else t[half][m | s] = got;
          }
    }
  }
  if (!rec) return;
  uint32_t m01 = 0xffffffffu, m23 = 0xffffffffu;   // bytes of the tokens 2b, 2b+1 | 2b+8, 2b+9 that are new
  if (FMT == 8 && keep > 0) {
    const int b = lane & 3;
    m01 = (2 * b >= keep ? 0x00ff00ffu : 0u) | (2 * b + 1 >= keep ? 0xff00ff00u : 0u);
    m23 = (2 * b + 8 >= keep ? 0x00ff00ffu : 0u) | (2 * b + 9 >= keep ? 0xff00ff00u : 0u);
  }
#pragma unroll
  for (int kp = 0; kp < 4; ++kp) {
    uint32_t w[4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int m = 2 * kp + u;
      // INT8: channel m of chunks a and a + 8; FP8: channel a of chunks 2m and 2m + 1
      const uint32_t x = FMT == kI8 ? t[0][m] : t[m >> 2][(2 * m) & 7], y = FMT == kI8 ? t[1][m] : t[m >> 2][(2 * m + 1) & 7];
      w[2 * u] = __byte_perm(x, y, 0x5410);
      w[2 * u + 1] = __byte_perm(x, y, 0x7632);
    }
    uint4* dst = reinterpret_cast<uint4*>(rec + R8::kVc + kp * 512 + lane * 16);
    uint4 z = make_uint4(w[0], w[1], w[2], w[3]);
    if (FMT == 8 && keep > 0) z = blend(z, *dst, m01, m23, m01, m23);
    *dst = z;
  }
}

template <int FMT, int DT>
__device__ __forceinline__ void put_keys(char* rec, const uint4 (&k)[8], const Coder& cd, int keep) {
  if (FMT == 8 && !power_of_two(cd.s)) put_keys_by<FMT, DT, false>(rec, k, cd, keep);
  else put_keys_by<FMT, DT, true>(rec, k, cd, keep);
}
template <int FMT, int DT>
__device__ __forceinline__ void put_values(char* rec, const uint4 (&v)[8], const Coder& cd, int keep) {
  if (FMT == 8 && !power_of_two(cd.s)) put_values_by<FMT, DT, false>(rec, v, cd, keep);
  else put_values_by<FMT, DT, true>(rec, v, cd, keep);
}

// Chunk c's partner chunk in a row spread over eight lanes as put_keys has it (lo:
// chunks 0..7 by lane, hi: 8..15).
__device__ __forceinline__ uint4 partner_chunk(const RopeArgs& r, int c, uint4 lo, uint4 hi) {
  const int p = rope::partner(r, c), from = (threadIdx.x & 24) | (p & 7);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t x = __shfl_sync(0xffffffffu, word(lo, i), from), y = __shfl_sync(0xffffffffu, word(hi, i), from);
    w[i] = p < 8 ? x : y;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A block's keys (tokens t0 + first .. t0 + last) turned by their positions.
template <int DT>
__device__ __forceinline__ void turn_keys(const RopeArgs& r, uint4 (&k)[8], int t0, int first, int last) {
  const int lane = threadIdx.x & 31, kc = lane & 7, kr = lane >> 3;
  if (r.interleaved || r.dim == kD) {
    // a lane's chunks c and c + 8 are a unit of the rotation; the next row's angles
    // load while this one turns. (Rows past `last` may lie past the table.)
    rope::Unit u[2];
    rope::unit_chunks(r, kc, u[0]);
    u[1] = u[0];
    rope::unit_angles(r, t0 + min(kr, last), u[0]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i < 3) rope::unit_angles(r, t0 + min(4 * (i + 1) + kr, last), u[(i + 1) & 1]);
      if (4 * i + kr >= first && 4 * i + kr <= last) rope::turn_unit<DT>(r, u[i & 1], k[2 * i], k[2 * i + 1]);
    }
  } else {   // a pair's other chunk is another lane's
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int x = 4 * i + kr;
      const uint4 lo = k[2 * i], hi = k[2 * i + 1];
      const uint4 plo = partner_chunk(r, kc, lo, hi), phi = partner_chunk(r, kc + 8, lo, hi);
      if (x >= first && x <= last) {
        k[2 * i] = rope::turn(r, t0 + x, kc, lo, plo, DT);
        k[2 * i + 1] = rope::turn(r, t0 + x, kc + 8, hi, phi, DT);
      }
    }
  }
}

struct Seq {
  int i, slot, T0, T1, c0;
  bool ok;
  // whole pages of new tokens, by logical page: [first_page, end_page)
  __device__ __forceinline__ int first_page() const { return (T0 + kP - 1) / kP; }
  __device__ __forceinline__ int end_page() const { return T1 / kP; }
  __device__ __forceinline__ int pages() const { return max(0, end_page() - first_page()); }
};

// Sequence i's row range, lengths and slot, checked but for the stored length; errors
// are reported by the keys' edge items (tell), all of a sequence's items agree on them.
template <bool ROPE>
__device__ __forceinline__ Seq sequence(const AppendArgs& a, int i, bool tell) {
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
  }
  s.ok = bad == 0;
  if (bad && tell && (threadIdx.x & 31) == 0) report(a.status, S4KV_ERR_DEVICE, bad, arg);
  return s;
}

template <int FMT>
__device__ __forceinline__ char* record(const AppendArgs& a, int pp, int h) {
  if (pp < 0 || pp >= a.num_pages) {
    if ((threadIdx.x & 31) == 0) report(a.status, S4KV_ERR_DEVICE, S4KV_DEV_BAD_PAGE, pp);
    return nullptr;
  }
  return a.pages + (static_cast<long long>(pp) * a.H + h) * Rec<FMT>::kBytes;
}

// Rows of a block's keys and values that this lane loads: token (row) of piece i.
__device__ __forceinline__ int key_row(int i) { return 4 * (i >> 1) + ((threadIdx.x & 31) >> 3); }
__device__ __forceinline__ int key_chunk(int i) { return (threadIdx.x & 7) + 8 * (i & 1); }
__device__ __forceinline__ int value_row(int i) { return 2 * (threadIdx.x & 3) + ((i >> 1) & 1) + 8 * (i >> 2); }
__device__ __forceinline__ int value_chunk(int i) { return ((threadIdx.x & 31) >> 2) + 8 * (i & 1); }

// One tensor of a block whose rows do not all come from the input: rows x < first
// are ring rows (INT8, keys already turned) or stay as they are in the record (FP8),
// rows [first, last] are the input's, later ones are absent (FP8: zeros, past the
// sequence's length).
template <int FMT, int DT, bool ROPE>
__device__ __forceinline__ void mixed_block(const AppendArgs& a, const Seq& s, int h, bool values, int page, int first, int last) {
  const int t0 = page * kP;
  const long long step = static_cast<long long>(a.H) * kD;
  const uint16_t* in = (values ? a.v : a.k) + (static_cast<long long>(s.c0 + t0 - s.T0) * a.H + h) * kD;   // token t0's row (used from `first` on)
  const uint16_t* ring = values ? reinterpret_cast<const uint16_t*>(a.vring) + s.slot * a.vring_slot + h * a.vring_head
                                : reinterpret_cast<const uint16_t*>(a.kring) + s.slot * a.kring_slot + h * a.kring_head;
  char* rec = record<FMT>(a, a.block_table[static_cast<long long>(s.i) * a.bt_stride + page], h);
  uint4 x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = values ? value_row(i) : key_row(i), c = values ? value_chunk(i) : key_chunk(i);
    x[i] = make_uint4(0u, 0u, 0u, 0u);
    if (r >= first && r <= last) x[i] = reinterpret_cast<const uint4*>(in + r * step)[c];
    else if (FMT == kI8 && r < first) x[i] = reinterpret_cast<const uint4*>(ring + r * kD)[c];
  }
  if (ROPE && !values) turn_keys<DT>(a.rope, x, t0, first, last);
  const Coder cd = coder<FMT, DT>(x, FMT == 8 ? a.fp8_scale[values ? a.H + h : h] : 0.0f);
  if (values) put_values<FMT, DT>(rec, x, cd, first);
  else if (rec) put_keys<FMT, DT>(rec, x, cd, first);
  if (FMT == kI8 && rec && (threadIdx.x & 31) == 0) *reinterpret_cast<float*>(rec + (values ? R8::kVs : R8::kKs)) = cd.s;
  __syncwarp();   // every lane has read its ring rows
}

// FP8: one token of one tensor into its record, lane l its channels 4l .. 4l+3.
template <int DT, bool ROPE>
__device__ __forceinline__ void fp8_token(const AppendArgs& a, const Seq& s, int h, bool values, int t, char* rec) {
  const int lane = threadIdx.x & 31, tau = t % kP;
  const uint16_t* row = (values ? a.v : a.k) + (static_cast<long long>(s.c0 + t - s.T0) * a.H + h) * kD;
  uint2 x = reinterpret_cast<const uint2*>(row)[lane];
  if (ROPE && !values) {   // lanes 2c and 2c + 1 share chunk c; each keeps its half
    const uint4 y = rope::turned_chunk(a.rope, row, t, lane >> 1, DT);
    x = (lane & 1) ? make_uint2(y.z, y.w) : make_uint2(y.x, y.y);
  }
  Coder cd;
  cd.s = a.fp8_scale[values ? a.H + h : h];
  cd.inv = 0.0f;
  const uint32_t lo = code_pair<8, DT, false>(x.x, cd), hi = code_pair<8, DT, false>(x.y, cd);
  if (!values) {   // slice kk = l % 8, column b = l / 8
    char* dst = rec + R8::kKc + ((lane & 7) >> 1) * 512 + (4 * (tau & 7) + (lane >> 3)) * 16 + 8 * (lane & 1) + 2 * (tau >> 3);
    *reinterpret_cast<uint16_t*>(dst) = static_cast<uint16_t>(lo);
    *reinterpret_cast<uint16_t*>(dst + 4) = static_cast<uint16_t>(hi);
  } else {         // channel 4l + q = 16 mt + a + 8 up; token 2b + r + 8w
    const int mt = lane >> 2, up = (lane >> 1) & 1, b = (tau & 7) >> 1;
    char* dst = rec + R8::kVc + (mt >> 1) * 512 + (4 * (4 * (lane & 1)) + b) * 16 + 8 * (mt & 1) + 4 * (tau >> 3) + 2 * up + (tau & 1);
    dst[0] = static_cast<char>(lo);
    dst[64] = static_cast<char>(lo >> 8);
    dst[128] = static_cast<char>(hi);
    dst[192] = static_cast<char>(hi >> 8);
  }
}

// FP8: new tokens [t0, t1) of one page. Few go one by one (a whole block is some
// thousand instructions of one warp), more as a block.
constexpr int kFewTokens = 4;
template <int DT, bool ROPE>
__device__ __forceinline__ void fp8_part(const AppendArgs& a, const Seq& s, int h, bool values, int t0, int t1) {
  const int page = t0 / kP;
  if (t1 - t0 > kFewTokens) {
    mixed_block<8, DT, ROPE>(a, s, h, values, page, t0 - page * kP, t1 - 1 - page * kP);
    return;
  }
  char* rec = record<8>(a, a.block_table[static_cast<long long>(s.i) * a.bt_stride + page], h);
  if (!rec) return;
  for (int t = t0; t < t1; ++t) fp8_token<DT, ROPE>(a, s, h, values, t, rec);
}

// Whether x holds for a thread of warps 2 (ID - 1) and 2 (ID - 1) + 1: both come here.
template <int ID>
__device__ __forceinline__ bool pair_or(bool x) {
  int y = x;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.s32 p, %0, 0;\n\tbarrier.cta.red.or.pred p, %1, 64, p;\n\t"
      "selp.s32 %0, 1, 0, p;\n\t}"
      : "+r"(y)
      : "n"(ID)
      : "memory");
  return y != 0;
}

// The edge of (sequence, head, tensor): see the top of the file. Keys and values are
// two neighbouring warps (pair x is warps 2x and 2x + 1); the keys' reports errors, looks
// at the stored length for both and stores the new one.
template <int FMT, int DT, bool ROPE>
__device__ __forceinline__ void edge(const AppendArgs& a, int i, int h, bool values) {
  const int lane = threadIdx.x & 31;
  const Seq s = sequence<ROPE>(a, i, !values);
  int* len = a.lens + s.slot * a.H + h;
  // with whole pages too the length is every item's to count (a slot that starts afresh
  // may have held any length: nothing to look at)
  const bool shared_len = s.T0 != 0 && s.pages() > 0;
  bool go = false;
  if (!values && lane == 0) {
    go = s.ok;
    if (go && s.T0 != 0) {
      go = shared_len ? goes_on(len, s.T0) : __ldcg(len) == s.T0;
      if (!go) report(a.status, S4KV_ERR_DEVICE, S4KV_DEV_BAD_LENGTH, i);
    }
  }
  go = threadIdx.x < 64 ? pair_or<1>(go) : pair_or<2>(go);
  if (!go) return;
  const int head = s.T0 % kP, end = s.T1 - s.T1 % kP;
  if constexpr (FMT == 8) {
    // the page that earlier and new tokens share, then a last page that is not full
    if (head != 0 && s.T1 > s.T0) fp8_part<DT, ROPE>(a, s, h, values, s.T0, min(s.T1, s.T0 - head + kP));
    if (s.T1 > end && end >= s.T0) fp8_part<DT, ROPE>(a, s, h, values, end, s.T1);
  } else {
    if (head != 0 && s.T0 - head + kP <= s.T1) mixed_block<FMT, DT, ROPE>(a, s, h, values, s.T0 / kP, head, kP - 1);
    // tokens [max(T0, last block), T1) wait in the rings
    const int from = max(s.T0, end), n = s.T1 - from;
    const uint16_t* in = (values ? a.v : a.k) + (static_cast<long long>(s.c0 + from - s.T0) * a.H + h) * kD;
    uint16_t* ring = values ? reinterpret_cast<uint16_t*>(a.vring) + s.slot * a.vring_slot + h * a.vring_head
                            : reinterpret_cast<uint16_t*>(a.kring) + s.slot * a.kring_slot + h * a.kring_head;
#pragma unroll 4
    for (int q = lane; q < 16 * n; q += 32) {
      const int t = from + (q >> 4), c = q & 15;
      const uint16_t* row = in + static_cast<long long>(q >> 4) * a.H * kD;
      uint4 x;
      if (ROPE && !values) x = rope::turned_chunk(a.rope, row, t, c, DT);
      else x = reinterpret_cast<const uint4*>(row)[c];
      reinterpret_cast<uint4*>(ring + (t % kP) * kD)[c] = x;
    }
  }
  if (!values && lane == 0) {
    if (shared_len) looked(len, s.T0, s.T1, 1, s.pages() + 1);
    else __stcg(len, s.T1);
  }
}

__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src)
               : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void all_but_newest_group() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }

// A page of new tokens on its way through a warp.
struct Page {
  int t0, pp, h;         // first token, pool page, kv head
  long long at;          // element offset of its first row in the input
};

template <int FMT, int DT, bool ROPE>
__global__ void __launch_bounds__(kThreads, kCtas) append8_kernel(AppendArgs a) {
  stream_wait();
  extern __shared__ __align__(128) uint8_t smem_raw[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint4* mine = reinterpret_cast<uint4*>(smem_raw + warp * kStage) + lane;   // piece i of this lane at mine[32 i]
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
  // Page slots: the page of new tokens whose first input row is x has slot
  // ceil(x / 16). Pages of a sequence are 16 rows apart and the next sequence starts
  // past the last one's 16 rows, so slots are distinct, and row 16 slot lies inside
  // the page: it names the sequence.
  const int slots = a.step ? 0 : (a.num_new + kP - 1) / kP;
  const int ctas = static_cast<int>(gridDim.x) - a.query_ctas;
  if constexpr (ROPE) {
    if (static_cast<int>(blockIdx.x) >= ctas) {
      const long long items = rope::query_items(a.rope, a.num_new), step = static_cast<long long>(a.query_ctas) * kWarps;
      for (long long q = static_cast<long long>(warp) * a.query_ctas + (blockIdx.x - ctas); q < items; q += step)
        rope::query_item<DT>(a, q);
      return;
    }
  }
  const long long stride = static_cast<long long>(ctas) * kWarps;
  const long long w0 = static_cast<long long>(blockIdx.x) * kWarps + warp;
  // the edges go to the warps that have the fewest pages, from the last one down: warps 2x
  // and 2x + 1 of a CTA have the values and the keys of the same ones, in step
  const long long edges = 2LL * a.n * a.H;
  for (long long e = stride - 1 - w0; e < edges; e += stride) {
    const long long sh = e >> 1;
    edge<FMT, DT, ROPE>(a, static_cast<int>(sh / a.H), static_cast<int>(sh % a.H), e & 1);
  }
  {
    // Page items (slot, head), head by head within a slot. A warp has one head and
    // neighbouring slots where the heads divide the warps (so that few sequences' lengths
    // are looked at and counted: 16000 tokens behind 1000 of each of 8 sequences 19.5 us,
    // slots all warps apart 25), else whatever comes: the next one is dslot and dhead on.
    int slot = static_cast<int>(w0) / a.H, h = static_cast<int>(w0) - slot * a.H, end = slots, dslot = a.dslot;
    if (a.dhead == 0) {
      const int x = slot, more = slots - a.each * a.dslot;   // the first `more` warps of a head have one more
      slot = x * a.each + min(x, more);
      end = slot + a.each + (x < more ? 1 : 0);
      dslot = 1;
    }
    Seq s;   // the sequence of the last page looked at
    s.i = -1;
    int sh = -1, c1 = 0;
    bool ask = false;   // whether s has still to be looked at
    int owed = 0;       // the pages that it has just been looked at for
    // the next page of this warp, from item (slot, h) on, which moves past it
    auto next = [&](Page& p) -> bool {
      while (slot < end) {
        const int row = slot * kP, hh = h, left = end - slot;   // (left: of this warp, where it has one head)
        slot += dslot;
        h += a.dhead;
        if (h >= a.H) {
          h -= a.H;
          ++slot;
        }
        if (s.i < 0 || hh != sh || row < s.c0 || row >= c1) {
          s = sequence<ROPE>(a, rope::sequence_of_row(a.cu_new, a.n, row), false);
          c1 = s.c0 + (s.T1 - s.T0);
          sh = hh;
          ask = s.T0 != 0;
        }
        const int page = (s.T0 + row - s.c0) / kP;
        if (!s.ok || page < s.first_page() || page >= s.end_page()) continue;
        if (ask) {   // for all of this warp's pages of (sequence, head)
          ask = false;
          s.ok = goes_on(a.lens + s.slot * a.H + hh, s.T0);
          if (!s.ok) continue;
          owed = a.dhead == 0 ? min(s.end_page() - page, left) : 1;
        }
        p.t0 = page * kP;
        p.h = hh;
        p.at = (static_cast<long long>(s.c0 + p.t0 - s.T0) * a.H + hh) * kD;
        p.pp = a.block_table[static_cast<long long>(s.i) * a.bt_stride + page];
        return true;
      }
      return false;
    };
    const long long step = static_cast<long long>(a.H) * kD;
    auto load_keys = [&](const Page& p) {
#pragma unroll
      for (int i = 0; i < 8; ++i) copy16(mine + 32 * i, a.k + p.at + key_row(i) * step + 8 * key_chunk(i));
    };
    auto load_values = [&](const Page& p) {
#pragma unroll
      for (int i = 0; i < 8; ++i) copy16(mine + 32 * (8 + i), a.v + p.at + value_row(i) * step + 8 * value_chunk(i));
    };
    auto pay = [&]() {   // (behind the loads of the page that next found)
      if (owed > 0 && lane == 0) looked(a.lens + s.slot * a.H + sh, s.T0, s.T1, owed, s.pages() + 1);
      owed = 0;
    };
    Page cur, nxt;
    bool have = next(cur);
    if (have) load_keys(cur);
    copies_end();
    if (have) load_values(cur);
    copies_end();
    pay();
    while (have) {
      const bool more = next(nxt);
      char* rec = record<FMT>(a, cur.pp, cur.h);
      uint4 x[8];
      all_but_newest_group();   // the keys are there
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = mine[32 * i];
      if constexpr (ROPE) turn_keys<DT>(a.rope, x, cur.t0, 0, kP - 1);
      const Coder kc = coder<FMT, DT>(x, FMT == 8 ? a.fp8_scale[cur.h] : 0.0f);
      if (more) load_keys(nxt);   // (x holds this page's)
      copies_end();
      if (rec) put_keys<FMT, DT>(rec, x, kc, 0);
      all_but_newest_group();   // the values are there
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = mine[32 * (8 + i)];
      const Coder vc = coder<FMT, DT>(x, FMT == 8 ? a.fp8_scale[a.H + cur.h] : 0.0f);
      if (more) load_values(nxt);
      copies_end();
      pay();
      put_values<FMT, DT>(rec, x, vc, 0);
      if (FMT == kI8 && rec && lane == 0) *reinterpret_cast<float2*>(rec + R8::kKs) = make_float2(kc.s, vc.s);
      cur = nxt;
      have = more;
    }
  }
}

template <int FMT>
cudaError_t run(const AppendArgs& a, int num_sms, cudaStream_t st) {
  const bool turn = a.rope.table != nullptr, bf = a.dtype == S4KV_BF16;
  void (*f)(AppendArgs);
  if constexpr (FMT == 8) f = bf ? append8_kernel<8, S4KV_BF16, true> : append8_kernel<8, S4KV_F16, true>;
  else if (turn) f = bf ? append8_kernel<kI8, S4KV_BF16, true> : append8_kernel<kI8, S4KV_F16, true>;
  else f = bf ? append8_kernel<kI8, S4KV_BF16, false> : append8_kernel<kI8, S4KV_F16, false>;
  const cudaError_t c = prefer_max_shared(reinterpret_cast<const void*>(f));
  if (c != cudaSuccess) return c;
  const long long slots = a.step ? 0 : (a.num_new + kP - 1) / kP;
  const long long items = slots * a.H + 2LL * a.n * a.H, queries = rope::query_items(a.rope, a.num_new);
  const long long cap = static_cast<long long>(num_sms) * kCtas;
  long long grid = min(cap, (items + kWarps - 1) / kWarps), more = (queries + kWarps - 1) / kWarps;
  if (grid + more > cap && more > 0) {   // divide a resident wave by the time that each kind takes
    more = min(more, max(cap * queries / (queries + kPageQueries * items), 1LL));
    grid = min(grid, max(cap - more, 1LL));
  }
  // whole multiples of the heads over the warps: a warp keeps its head from page to page
  int unit = a.H;
  while (unit % 2 == 0 && unit * kWarps / 2 % a.H == 0) unit /= 2;
  if (grid > unit) grid -= grid % unit;
  AppendArgs b = a;
  b.query_ctas = static_cast<int>(more);
  b.dslot = static_cast<int>(grid * kWarps / a.H);
  b.dhead = static_cast<int>(grid * kWarps % a.H);
  b.each = b.dslot > 0 ? static_cast<int>(slots / b.dslot) : 0;
  return launch_behind(f, dim3(static_cast<unsigned>(grid + more)), dim3(kThreads), kWarps * kStage, st, b);
}

}  // namespace

cudaError_t launch_append8(const AppendArgs& a, int num_sms, cudaStream_t st) {
  if (a.bits == kI8) return run<kI8>(a, num_sms, st);
  if (a.bits != 8 || !a.rope.table) return cudaErrorInvalidValue;
  return run<8>(a, num_sms, st);
}

}  // namespace s4kv
