// Restoring tokens from page records and rings, in registers (s4kv_gather.cu: into dense
// rows; s4kv_tiles.cu: into tiles of matrix operands). One warp, one tensor of one page (or
// key group) of one kv head, straight from the record's words. `put(token, c, y)` takes
// channels 8c .. 8c + 7 of a token, the first token of the page (or group) being 0. `fp8_scale`
// points to the tensor's scale of the head on FP8 pages and is not looked at on others.
//
// Keys: lane l takes chunk c = l % 8 and c + 8 of 8 channels of tokens 4i + l / 8 and + 8,
// whose words hold both tokens. Values: lane (a, b) = (l / 4, l % 4) takes chunks a and
// a + 8 of tokens 2b, 2b+1, 2b+8, 2b+9; an INT8 lane's words hold just these, the others'
// hold channel a of every chunk, and an 8 x 8 transpose over the lanes of one b brings
// them there.
//
// For translation units compiled without FMA contraction: a restored value is
// fmaf(code, scale, min) (KIVI) or code * scale (8-bit).
#pragma once

#include "s4kv_common.cuh"

#include <cuda_fp8.h>

namespace s4kv {
namespace {

constexpr int kI8 = S4KV_BITS_INT8;
template <int FMT> constexpr bool kByte = FMT == 8 || FMT == kI8;

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

// Tokens [lo, hi) (of 0..15, token 0 at position t0) from ring rows t % mod: every load first.
template <class PUT>
__device__ __forceinline__ void put_ring(const uint16_t* ring, int mod, int t0, int lo, int hi, int dtype, const PUT& put) {
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
    put(tau, c, y);
  }
}

// Tokens [lo, hi) of the keys of an 8-bit page's record.
template <int FMT, class PUT>
__device__ __forceinline__ void put_keys(const float* fp8_scale, const char* rec, int lo, int hi, const PUT& put) {
  const int lane = threadIdx.x & 31, kr = lane >> 3, kc = lane & 7;
  uint4 w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = key_words<FMT>(rec, 4 * (i >> 1) + kr, kc + 8 * (i & 1));
  float ks;
  if constexpr (FMT == kI8) ks = *reinterpret_cast<const float*>(rec + Rec<kI8>::kKs);
  else ks = *fp8_scale;
  const float s8[8] = {ks}, none[8] = {};
#pragma unroll
  for (int half = 0; half < 2; ++half)
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int tau = 4 * (x >> 1) + kr + 8 * (x & 1);
      if (tau < lo || tau >= hi) continue;
      float y[8];
      keys8<FMT>(w[2 * (x >> 1) + half], x & 1, s8, none, y);
      put(tau, kc + 8 * half, y);
    }
}

// A whole key group (KIVI): tokens [lo, hi) (of 0..31) of its two pages, whose records
// hold the metadata of channels 0..63 and 64..127 for both.
template <int FMT, class PUT>
__device__ __forceinline__ void put_key_group(const char* rec0, const char* rec1, int lo, int hi, const PUT& put) {
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
        put(t, c, y);
      }
  }
}

// Tokens [lo, hi) of the values of a record.
template <int FMT, class PUT>
__device__ __forceinline__ void put_values(const float* fp8_scale, const char* rec, int lo, int hi, const PUT& put) {
  const int lane = threadIdx.x & 31, ca = lane >> 2, b = lane & 3;
  uint4 v[kValueWords<FMT>];
  value_words<FMT>(rec, v);
  float vs = 0.0f;
  float4 s4[2], m4[2];   // KIVI, by half: of tokens 2b, 2b+1, 2b+8, 2b+9
  if constexpr (FMT == kI8) vs = *reinterpret_cast<const float*>(rec + Rec<kI8>::kVs);
  else if constexpr (FMT == 8) vs = *fp8_scale;
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
      put(tau, ca + 8 * half, y);
    }
}

}  // namespace
}  // namespace s4kv
