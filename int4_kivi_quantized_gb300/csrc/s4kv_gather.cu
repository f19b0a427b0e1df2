// Batched restore (s4kv_gather): token ranges of many sequences out of the pages
// and rings into dense rows, for every page format. One pass over the records that
// the ranges need and one over the rows: bound by those bytes.
//
// Work item, one warp: one tensor of one page of one kv head (keys and values apart
// leave registers for twice the warps), straight from the record's words
// (in the order of the attention kernels' operands) to rows, in registers. Keys:
// lane l takes chunk c = l % 8 and c + 8 of 8 channels of tokens 4i + l / 8 and + 8,
// whose words hold both tokens, so a store instruction writes 128 contiguous bytes
// of four rows. Values: lane (a, b) = (l / 4, l % 4) takes chunks a and a + 8 of
// tokens 2b, 2b+1, 2b+8, 2b+9; an INT8 lane's words hold just these, the others'
// hold channel a of every chunk, and an 8 x 8 transpose over the lanes of one b
// brings them there.
//
// Measured (8 prompts of 1900 to 2048 tokens, 8 kv heads, into 16-bit rows; bytes at a
// plain copy's 6783 GB/s): INT8 and FP8 16.5 us (bytes 14.3), 4-bit 17.7 (13.1), 2-bit 16
// (11.9); histories of 336 MB of rows 96.8 (74.3; a fill of those rows alone 84: writes go
// slower than copies), of 671 MB of fp32 rows 181 (124). 300000 tokens x heads with 1, 2, 5 and
// 8 kv heads: 4-bit 58, 57, 57, 47 (31), 2-bit 56, 54, 54, 43 (28), INT8 46, 46, 57, 48 (34):
// with one or two heads the 4- and 2-bit key warps of every other page have nothing to do (a
// group goes with its first page), with five some of the second row of CTAs.
//
// Page slots: sequence i starts at slot cu_rows[i] / 16 + 2 i; a range of x rows
// touches at most x / 16 + 2 pages, so sequences do not overlap, and a slot finds
// its sequence by a search over cu_rows alone.
//
// Compiled without FMA contraction: a restored value is fmaf(code, scale, min)
// (KIVI) or code * scale (8-bit), rounded once more only to a 16-bit out_dtype.

#include "s4kv_common.cuh"

#include <cuda_fp8.h>
#include <type_traits>

namespace s4kv {
namespace {

constexpr int kI8 = S4KV_BITS_INT8;
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
// (two or three of them, on the prompts above: INT8 16.6 / 19.4 us, 4-bit 17.8 / 27.2: at 80
// registers a lane keeps fewer loads in flight)
#ifndef S4KV_GATHER_CTAS
#define S4KV_GATHER_CTAS 2
#endif
constexpr int kCtas = S4KV_GATHER_CTAS;   // resident CTAs per SM the registers are budgeted for
template <int FMT> constexpr bool kByte = FMT == 8 || FMT == kI8;

// Eight channels at element `at` of an output tensor.
template <typename OUT>
__device__ __forceinline__ void put8(OUT* at, const float (&y)[8]) {
  if constexpr (std::is_same_v<OUT, float>) {
    reinterpret_cast<float4*>(at)[0] = make_float4(y[0], y[1], y[2], y[3]);
    reinterpret_cast<float4*>(at)[1] = make_float4(y[4], y[5], y[6], y[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (std::is_same_v<OUT, __nv_bfloat16>) {
        const __nv_bfloat162 x = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&x);
      } else {
        const __half2 x = __floats2half2_rn(y[2 * i], y[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&x);
      }
    }
    *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// A chunk of 16-bit values, widened exactly.
__device__ __forceinline__ void widen8(uint4 v, int dtype, float (&y)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[2 * i] = widen16(static_cast<uint16_t>(w[i] & 0xffff), dtype);
    y[2 * i + 1] = widen16(static_cast<uint16_t>(w[i] >> 16), dtype);
  }
}

// Byte i of w as a number less `offset`: 2^23 + n has n in its low mantissa bits.
__device__ __forceinline__ float byte_number(uint32_t w, int i, float offset) {
  return __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440 + i)) - (8388608.0f + offset);
}
// Two e4m3 bytes, low first.
__device__ __forceinline__ float2 e4m3x2(uint32_t w) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w & 0xffffu), __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Records are read by plain loads: the work before this kernel may still be writing them
// when it starts, so they are not constant over its lifetime.

// The key words of chunk c of tokens ta and ta + 8: 8-bit pages 16 bytes, 4-bit 8
// bytes (slices 2 (c % 4) and + 1), 2-bit 4 bytes.
template <int FMT>
__device__ __forceinline__ uint4 key_words(const char* rec, int ta, int c) {
  const int L = 4 * ta + (c >> 2), j = c & 3;
  if constexpr (kByte<FMT>) {
    return *reinterpret_cast<const uint4*>(rec + j * 512 + L * 16);
  } else if constexpr (FMT == 4) {
    const uint2 w = *reinterpret_cast<const uint2*>(rec + Rec<4>::kKc + (j >> 1) * 512 + L * 16 + (j & 1) * 8);
    return make_uint4(w.x, w.y, 0u, 0u);
  } else {
    return make_uint4(*reinterpret_cast<const uint32_t*>(rec + Rec<2>::kKc + L * 16 + j * 4), 0u, 0u, 0u);
  }
}

// The chunk's eight keys of token ta + 8 hi: s the scales (8-bit: s[0]) and m the
// minima of its channels.
template <int FMT>
__device__ __forceinline__ void keys8(uint4 w, int hi, const float (&s)[8], const float (&m)[8], float (&y)[8]) {
  if constexpr (kByte<FMT>) {
    const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      float2 f;
      if constexpr (FMT == kI8) f = make_float2(byte_number(q[x], 2 * hi, 128.0f), byte_number(q[x], 2 * hi + 1, 128.0f));
      else f = e4m3x2(q[x] >> (16 * hi));
      y[2 * x] = __fmul_rn(f.x, s[0]);
      y[2 * x + 1] = __fmul_rn(f.y, s[0]);
    }
  } else {
#pragma unroll
    for (int half = 0; half < 2; ++half) {   // bytes c_0, c_2, c_1, c_3 of four channels
      uint32_t q;
      if constexpr (FMT == 4) q = ((half ? w.y : w.x) >> (4 * hi)) & 0x0f0f0f0fu;
      else q = (w.x >> (2 * (2 * half + hi))) & 0x03030303u;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int at = e == 1 ? 2 : e == 2 ? 1 : e;
        y[4 * half + e] = __fmaf_rn(byte_number(q, at, 0.0f), s[4 * half + e], m[4 * half + e]);
      }
    }
  }
}

// Scales and minima of key chunk c from the record of the page of the pair that
// holds them.
template <int FMT>
__device__ __forceinline__ void key_meta(const char* meta, int c, float (&s)[8], float (&m)[8]) {
  using F = Rec<FMT>;
  const int u = (c >> 2) & 1, i = 2 * (c & 3);
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const float4* p = reinterpret_cast<const float4*>(meta + F::kKm + (2 * (i + half) + u) * 16);
    const float4 a = *p, b = *(p + 16);
    s[4 * half] = a.x; s[4 * half + 1] = a.y; s[4 * half + 2] = a.z; s[4 * half + 3] = a.w;
    m[4 * half] = b.x; m[4 * half + 1] = b.y; m[4 * half + 2] = b.z; m[4 * half + 3] = b.w;
  }
}

// This lane's value words: 8-bit pages 64 bytes, 4-bit 32, 2-bit 16.
template <int FMT> constexpr int kValueWords = kByte<FMT> ? 4 : FMT == 4 ? 2 : 1;
template <int FMT>
__device__ __forceinline__ void value_words(const char* rec, uint4 (&v)[kValueWords<FMT>]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < kValueWords<FMT>; ++i) v[i] = *reinterpret_cast<const uint4*>(rec + Rec<FMT>::kVc + i * 512 + lane * 16);
}

// Their codes: t[half][m] holds channel m of chunk a + 8 half, a byte a token (8-bit
// pages in the order 2b, 2b+1, 2b+8, 2b+9, KIVI 2b, 2b+8, 2b+1, 2b+9). Called by the
// whole warp.
template <int FMT>
__device__ __forceinline__ void value_codes(const uint4 (&v)[kValueWords<FMT>], uint32_t (&t)[2][8]) {
  const int lane = threadIdx.x & 31;
  if constexpr (kByte<FMT>) {
#pragma unroll
    for (int kp = 0; kp < 4; ++kp) {
      const uint32_t w[4] = {v[kp].x, v[kp].y, v[kp].z, v[kp].w};
#pragma unroll
      for (int u = 0; u < 2; ++u) {   // words: tokens 2b, 2b+1 of x, of y | tokens 2b+8, 2b+9 of x, of y
        const uint32_t x = __byte_perm(w[2 * u], w[2 * u + 1], 0x5410), y = __byte_perm(w[2 * u], w[2 * u + 1], 0x7632);
        const int m = 2 * kp + u;
        if constexpr (FMT == kI8) {   // channel m of chunks a and a + 8
          t[0][m] = x;
          t[1][m] = y;
        } else {                      // channel a of chunks 2m and 2m + 1
          t[m >> 2][(2 * m) & 7] = x;
          t[m >> 2][(2 * m + 1) & 7] = y;
        }
      }
    }
  } else if constexpr (FMT == 4) {    // word mt: chunks 2 mt (low nibbles) and 2 mt + 1
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const uint32_t w[4] = {v[half].x, v[half].y, v[half].z, v[half].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        t[half][2 * i] = w[i] & 0x0f0f0f0fu;
        t[half][2 * i + 1] = (w[i] >> 4) & 0x0f0f0f0fu;
      }
    }
  } else {                            // word mp: chunks 4 mp + q by position
    const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) t[i >> 1][4 * (i & 1) + q] = (w[i] >> (2 * q)) & 0x03030303u;
  }
  if constexpr (FMT != kI8) {
    // channel a of every chunk -> every channel of chunk a: exchange half of the
    // entries a step over the lanes of one b
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
}

// Tokens [lo, hi) (of 0..15, token 0 at position t0) from ring rows t % mod to the
// rows at `dst` (token 0's; a token is `step` elements): every load first.
template <typename OUT>
__device__ __forceinline__ void put_ring(const uint16_t* ring, int mod, int t0, int lo, int hi, int dtype, OUT* dst, int step) {
  const int lane = threadIdx.x & 31, c = lane & 15, r = lane >> 4, at = t0 % mod;
  uint4 v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int tau = 2 * i + r;
    int row = at + tau;
    if (mod < kP) row %= mod;
    else if (row >= mod) row -= mod;
    if (tau >= lo && tau < hi) v[i] = reinterpret_cast<const uint4*>(ring + static_cast<long long>(row) * kD)[c];
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int tau = 2 * i + r;
    if (tau < lo || tau >= hi) continue;
    float y[8];
    widen8(v[i], dtype, y);
    put8(dst + static_cast<long long>(tau) * step + 8 * c, y);
  }
}

// Tokens [lo, hi) of the keys of an 8-bit page's record.
template <int FMT, typename OUT>
__device__ __forceinline__ void put_keys(const GatherArgs& a, const char* rec, int lo, int hi, OUT* dst, int step, int h) {
  const int lane = threadIdx.x & 31, kr = lane >> 3, kc = lane & 7;
  uint4 w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = key_words<FMT>(rec, 4 * (i >> 1) + kr, kc + 8 * (i & 1));
  float ks;
  if constexpr (FMT == kI8) ks = *reinterpret_cast<const float*>(rec + Rec<kI8>::kKs);
  else ks = a.fp8_scale[h];
  const float s8[8] = {ks}, none[8] = {};
#pragma unroll
  for (int half = 0; half < 2; ++half)
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int tau = 4 * (x >> 1) + kr + 8 * (x & 1);
      if (tau < lo || tau >= hi) continue;
      float y[8];
      keys8<FMT>(w[2 * (x >> 1) + half], x & 1, s8, none, y);
      put8(dst + static_cast<long long>(tau) * step + 8 * (kc + 8 * half), y);
    }
}

// A whole key group (KIVI): tokens [lo, hi) (of 0..31) of its two pages, whose records
// hold the metadata of channels 0..63 and 64..127 for both.
template <int FMT, typename OUT>
__device__ __forceinline__ void put_key_group(const char* rec0, const char* rec1, int lo, int hi, OUT* dst, int step) {
  const int lane = threadIdx.x & 31, kr = lane >> 3, kc = lane & 7;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int c = kc + 8 * half;
    float s8[8], m8[8];
    key_meta<FMT>(half ? rec1 : rec0, c, s8, m8);
    uint4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = key_words<FMT>(i >> 1 ? rec1 : rec0, 4 * (i & 1) + kr, c);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int t = 16 * (i >> 1) + 4 * (i & 1) + kr + 8 * x;
        if (t < lo || t >= hi) continue;
        float y[8];
        keys8<FMT>(w[i], x, s8, m8, y);
        put8(dst + static_cast<long long>(t) * step + 8 * c, y);
      }
  }
}

// Tokens [lo, hi) of the values of a record.
template <int FMT, typename OUT>
__device__ __forceinline__ void put_values(const GatherArgs& a, const char* rec, int lo, int hi, OUT* dst, int step, int h) {
  const int lane = threadIdx.x & 31, ca = lane >> 2, b = lane & 3;
  uint4 v[kValueWords<FMT>];
  value_words<FMT>(rec, v);
  float vs = 0.0f;
  float4 s4[2], m4[2];   // KIVI, by half: of tokens 2b, 2b+1, 2b+8, 2b+9
  if constexpr (FMT == kI8) vs = *reinterpret_cast<const float*>(rec + Rec<kI8>::kVs);
  else if constexpr (FMT == 8) vs = a.fp8_scale[a.H + h];
  else {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int k = (ca + 8 * half) >> 2;
      s4[half] = *(reinterpret_cast<const float4*>(rec + Rec<FMT>::kVm + ((2 * k) * 4 + b) * 16));
      m4[half] = *(reinterpret_cast<const float4*>(rec + Rec<FMT>::kVm + ((2 * k + 1) * 4 + b) * 16));
    }
  }
  uint32_t tc[2][8];
  value_codes<FMT>(v, tc);
#pragma unroll
  for (int half = 0; half < 2; ++half)
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int tau = 2 * b + (x & 1) + 8 * (x >> 1);
      if (tau < lo || tau >= hi) continue;
      float y[8];
      if constexpr (FMT == kI8) {
#pragma unroll
        for (int m = 0; m < 8; ++m) y[m] = __fmul_rn(byte_number(tc[half][m], x, 128.0f), vs);
      } else if constexpr (FMT == 8) {
#pragma unroll
        for (int m = 0; m < 8; m += 2) {
          const float2 f = e4m3x2(__byte_perm(tc[half][m], tc[half][m + 1], 0x40 + 0x11 * x));
          y[m] = __fmul_rn(f.x, vs);
          y[m + 1] = __fmul_rn(f.y, vs);
        }
      } else {
        const int at = x == 1 ? 2 : x == 2 ? 1 : x;
        const float sx = x == 0 ? s4[half].x : x == 1 ? s4[half].y : x == 2 ? s4[half].z : s4[half].w;
        const float mx = x == 0 ? m4[half].x : x == 1 ? m4[half].y : x == 2 ? m4[half].z : m4[half].w;
#pragma unroll
        for (int m = 0; m < 8; ++m) y[m] = __fmaf_rn(byte_number(tc[half][m], at, 0.0f), sx, mx);
      }
      put8(dst + static_cast<long long>(tau) * step + 8 * (ca + 8 * half), y);
    }
}

__device__ __forceinline__ int slot_base(const GatherArgs& a, int i) { return a.cu_rows[i] / kP + 2 * i; }

// The last i with slot_base(i) <= s, 32 probes a round.
__device__ __forceinline__ int sequence_of(const GatherArgs& a, int s) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = a.n;
  while (hi - lo > 1) {
    const int gap = (hi - lo + 31) / 32;
    const int at = lo + gap * (lane + 1);
    const unsigned past = __ballot_sync(0xffffffffu, at >= hi || slot_base(a, at) > s);
    const int k = __ffs(past) - 1;
    const int nlo = lo + gap * k;
    hi = min(hi, nlo + gap);
    lo = nlo;
  }
  return lo;
}

// Warps of a CTA: `combos` = min(2 H, 8) of the (head, tensor) pairs (blockIdx.y says
// which) side by side on a page, so that a token's heads are written together, and
// 8 / combos neighbouring pages. A CTA walks a contiguous run of page slots: the
// range that a slot lies in changes with the sequence.
template <int FMT, typename OUT>
__global__ void __launch_bounds__(kThreads, kCtas) gather_kernel(GatherArgs a, int combos, int slots) {
  stream_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  {   // a malformed call: nothing is read or written
    int bad = a.cu_rows[0] != 0 || a.cu_rows[a.n] != a.num_rows;
    for (int i = threadIdx.x; i < a.n; i += kThreads) {
      const int f = a.first ? a.first[i] : 0;
      bad |= a.cu_rows[i + 1] < a.cu_rows[i] || f < 0 || f > (1 << 30) || a.cu_rows[i + 1] - a.cu_rows[i] > (1 << 30);
    }
    if (__syncthreads_or(bad)) {
      if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) report(a.status, S4KV_ERR_DEVICE, S4KV_DEV_BAD_CU, a.n);
      return;
    }
  }
  const int side = kWarps / combos;   // pages of a CTA at once
  const int pair = static_cast<int>(blockIdx.y) * combos + warp % combos, h = pair >> 1;
  const bool values = pair & 1;
  if (warp >= side * combos || h >= a.H) return;
  const int s0 = static_cast<int>(static_cast<long long>(slots) * blockIdx.x / gridDim.x);
  const int s1 = static_cast<int>(static_cast<long long>(slots) * (blockIdx.x + 1) / gridDim.x);
  int base = 0, end = -1;   // the slots of the current range
  int f = 0, cnt = 0, quant = 0, seq = 0;
  bool ok = false;
  const uint16_t* ring = nullptr;
  OUT* rows = nullptr;      // of token 0 of the sequence (this head)
  const int step = a.H * kD;
  constexpr int kKMod = FMT == kI8 ? kP : kG;
  const int vmod = FMT == kI8 ? kP : a.R;
  for (int s = s0 + warp / combos; s < s1; s += side) {
    if (s >= end) {   // (slots only grow)
      seq = sequence_of(a, s);
      f = a.first ? a.first[seq] : 0;
      const int c0 = a.cu_rows[seq], c1 = a.cu_rows[seq + 1];
      cnt = c1 - c0;
      base = c0 / kP + 2 * seq;
      end = seq + 1 < a.n ? c1 / kP + 2 * seq + 2 : 0x7fffffff;
      const int T = a.seq_lens[seq], slot = a.slot_ids ? a.slot_ids[seq] : seq;
      // first token of the key and of the value residual
      const int Tk = FMT == 8 ? T : FMT == kI8 ? T / kP * kP : T & ~(kG - 1);
      const int Tv = FMT == 8 ? T : FMT == kI8 ? Tk : max(0, T - a.R);
      quant = values ? Tv : Tk;
      const long long stop = static_cast<long long>(f) + cnt;
      // the metadata of a key group spans its two pages
      const long long table = !kByte<FMT> && stop <= Tk ? (stop + kG - 1) / kG * kG : stop;
      int bad = 0, arg = seq;
      if (slot < 0 || slot >= a.max_slots) {
        bad = S4KV_DEV_BAD_SLOT;
        arg = slot;
      } else if (T < 0 || a.lens[slot * a.H + h] != T) {
        bad = S4KV_DEV_BAD_LENGTH;
      } else if (stop > T) {
        bad = S4KV_DEV_BAD_POSITION;
      } else if (static_cast<long long>(a.bt_stride) * kP < table) {
        bad = S4KV_DEV_BAD_TABLE;
      }
      ok = bad == 0 && cnt > 0;
      if (bad && cnt > 0 && lane == 0) report(a.status, S4KV_ERR_DEVICE, bad, arg);
      if (ok) {
        ring = values ? reinterpret_cast<const uint16_t*>(a.vring) + slot * a.vring_slot + h * a.vring_head
                      : reinterpret_cast<const uint16_t*>(a.kring) + slot * a.kring_slot + h * a.kring_head;
        rows = static_cast<OUT*>(values ? a.out_v : a.out_k) + (static_cast<long long>(c0 - f) * a.H + h) * kD;
      }
    }
    const int page = f / kP + (s - base), t0 = page * kP;
    const int lo = max(f - t0, 0);
    int hi = min(f + cnt - t0, kP);
    if (!ok || hi <= lo) continue;
    // KIVI: the keys of a whole group go with its first page that the range holds
    const bool group = !kByte<FMT> && !values && t0 < quant;
    if (group) {
      if ((page & 1) && page != f / kP) continue;
      if (!(page & 1)) hi = min(f + cnt - t0, kG);
    }
    const char* rec = nullptr;
    const char* rec1 = nullptr;   // (group) its second page
    if (t0 + lo < quant) {
      const int* bt = a.block_table + static_cast<long long>(seq) * a.bt_stride;
      const int p0 = bt[group ? page & ~1 : page], p1 = group ? bt[page | 1] : p0;
      auto out = [&](int p) { return p < 0 || p >= a.num_pages; };
      if (out(p0) || out(p1)) {
        if (lane == 0) report(a.status, S4KV_ERR_DEVICE, S4KV_DEV_BAD_PAGE, out(p0) ? p0 : p1);
        continue;
      }
      rec = a.pages + (static_cast<long long>(p0) * a.H + h) * Rec<FMT>::kBytes;
      rec1 = a.pages + (static_cast<long long>(p1) * a.H + h) * Rec<FMT>::kBytes;
    }
    OUT* dst = rows + static_cast<long long>(t0) * step;
    if (group) {
      if constexpr (!kByte<FMT>) {
        const int odd = (page & 1) * kP;
        put_key_group<FMT>(rec, rec1, odd + lo, odd + hi, dst - static_cast<long long>(odd) * step, step);
      }
      continue;
    }
    const int held = min(max(quant - t0, lo), hi);   // tokens [lo, held) are in the record, [held, hi) in the ring
    if (held > lo) {
      if (values) put_values<FMT>(a, rec, lo, held, dst, step, h);
      else if constexpr (kByte<FMT>) put_keys<FMT>(a, rec, lo, held, dst, step, h);
    }
    if (FMT != 8 && hi > held) put_ring(ring, values ? vmod : kKMod, t0, held, hi, a.dtype, dst, step);
  }
}

// The debug restore of INT8 pages: one slot, one kv head and eight tokens a block,
// thread = channel.
__global__ void __launch_bounds__(kD) dequant_int8_kernel(DequantArgs a) {
  const int h = blockIdx.y, c = threadIdx.x, T = a.T, Tq = T / kP * kP;
  if (blockIdx.x == 0 && c == 0 && a.lens[a.slot * a.H + h] != T)
    report(a.status, S4KV_ERR_DEVICE, S4KV_DEV_BAD_LENGTH, a.slot);
  const uint16_t* kring = reinterpret_cast<const uint16_t*>(a.kring) + a.slot * a.kring_slot + h * a.kring_head;
  const uint16_t* vring = reinterpret_cast<const uint16_t*>(a.vring) + a.slot * a.vring_slot + h * a.vring_head;
  for (int t = blockIdx.x * 8; t < min(T, static_cast<int>(blockIdx.x) * 8 + 8); ++t) {
    const int tau = t % kP;
    float kv = 0.0f, vv = 0.0f;
    if (t >= Tq) {
      kv = widen16(kring[tau * kD + c], a.dtype);
      vv = widen16(vring[tau * kD + c], a.dtype);
    } else {
      const int pp = a.bt_row[t / kP];
      if (pp < 0 || pp >= a.num_pages) {
        if (c == 0) report(a.status, S4KV_ERR_DEVICE, S4KV_DEV_BAD_PAGE, pp);
      } else {
        const char* rec = a.pages + (static_cast<long long>(pp) * a.H + h) * Rec<kI8>::kBytes;
        const uint8_t* p = reinterpret_cast<const uint8_t*>(rec);
        const int a7 = tau & 7, w = tau >> 3, q = c >> 3, x = (c & 7) >> 1;
        const int kb = p[(q & 3) * 512 + (4 * a7 + (q >> 2)) * 16 + 4 * x + 2 * w + (c & 1)];
        const int m = c & 7, va = (c >> 3) & 7, hi = c >> 6;
        const int vb = p[Rec<kI8>::kVc + (m >> 1) * 512 + (4 * va + (a7 >> 1)) * 16 + 8 * (m & 1) + 4 * w + 2 * hi + (tau & 1)];
        kv = __fmul_rn(static_cast<float>(kb - 128), *reinterpret_cast<const float*>(rec + Rec<kI8>::kKs));
        vv = __fmul_rn(static_cast<float>(vb - 128), *reinterpret_cast<const float*>(rec + Rec<kI8>::kVs));
      }
    }
    a.out_k[(static_cast<long long>(h) * T + t) * kD + c] = kv;
    a.out_v[(static_cast<long long>(h) * T + t) * kD + c] = vv;
  }
}

template <int FMT, typename OUT>
cudaError_t run_out(const GatherArgs& a, int num_sms, cudaStream_t st) {
  void (*f)(GatherArgs, int, int) = gather_kernel<FMT, OUT>;
  const cudaError_t c = prefer_max_shared(reinterpret_cast<const void*>(f));
  if (c != cudaSuccess) return c;
  const int pairs = 2 * a.H, combos = pairs < kWarps ? pairs : kWarps, side = kWarps / combos;
  const int parts = (pairs + combos - 1) / combos;
  const int slots = a.num_rows / kP + 2 * a.n;
  const int want = (slots + side - 1) / side, cap = (num_sms * kCtas + parts - 1) / parts;
  const int grid = want < cap ? want : cap;   // one wave: a CTA's checks cost more than a longer run
  return launch_behind(f, dim3(static_cast<unsigned>(grid), static_cast<unsigned>(parts)), dim3(kThreads), 0, st,
                       a, combos, slots);
}
template <int FMT>
cudaError_t run(const GatherArgs& a, int num_sms, cudaStream_t st) {
  if (a.out_dtype == S4KV_F32) return run_out<FMT, float>(a, num_sms, st);
  if (a.out_dtype == S4KV_BF16) return run_out<FMT, __nv_bfloat16>(a, num_sms, st);
  return run_out<FMT, __half>(a, num_sms, st);
}

}  // namespace

cudaError_t launch_gather(const GatherArgs& a, int num_sms, cudaStream_t st) {
  switch (a.bits) {
    case kI8: return run<kI8>(a, num_sms, st);
    case 8: return run<8>(a, num_sms, st);
    case 2: return run<2>(a, num_sms, st);
    default: return run<4>(a, num_sms, st);
  }
}

cudaError_t launch_dequant_int8(const DequantArgs& a, cudaStream_t st) {
  dequant_int8_kernel<<<dim3((a.T + 7) / 8, a.H), kD, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace s4kv
