// Rotary position embedding of 16-bit rows, shared by the append kernels: an
// 8-channel chunk of a row turned by the angles of its position. Every product
// and sum is one binary32 rounding (no fused multiply-add) and the result is
// rounded once to the cache dtype, so the rows are those of a rotation done in
// 32-bit arithmetic before an ordinary append, bit for bit.
#pragma once

#include "s4kv_common.cuh"

namespace s4kv {
namespace rope {

__device__ __forceinline__ void widen8(uint4 w, int dtype, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = widen16(static_cast<uint16_t>(u[i] & 0xffff), dtype);
    x[2 * i + 1] = widen16(static_cast<uint16_t>(u[i] >> 16), dtype);
  }
}

__device__ __forceinline__ uint4 round8(const float (&x)[8], int dtype) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (dtype == S4KV_BF16) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// The 8 chunk-aligned floats of a table row from index i on.
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

// Chunk that holds the partners of chunk c's channels (c itself where none is
// needed: interleaved pairs, and channels past the rotated ones).
__device__ __forceinline__ int partner(const RopeArgs& r, int c) {
  const int half = r.dim >> 4;   // chunks of the first half
  if (r.interleaved || c >= 2 * half) return c;
  return c < half ? c + half : c - half;
}

// Chunk c (channels 8c .. 8c+7) of a row at position `pos`, turned: x is the
// chunk, y its partner chunk.
__device__ __forceinline__ uint4 turn(const RopeArgs& r, int pos, int c, uint4 x, uint4 y, int dtype) {
  if (8 * c >= r.dim) return x;
  const float* row = r.table + static_cast<long long>(pos) * r.dim;
  const int half = r.dim >> 1;
  float a[8], o[8];
  widen8(x, dtype, a);
  if (r.interleaved) {
    const float4 cs = __ldg(reinterpret_cast<const float4*>(row + 4 * c));
    const float4 sn = __ldg(reinterpret_cast<const float4*>(row + half + 4 * c));
    const float cc[4] = {cs.x, cs.y, cs.z, cs.w}, ss[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[2 * i] = __fsub_rn(__fmul_rn(a[2 * i], cc[i]), __fmul_rn(a[2 * i + 1], ss[i]));
      o[2 * i + 1] = __fadd_rn(__fmul_rn(a[2 * i + 1], cc[i]), __fmul_rn(a[2 * i], ss[i]));
    }
  } else {
    float b[8], cc[8], ss[8];
    widen8(y, dtype, b);
    const bool second = 8 * c >= half;
    const int i0 = second ? 8 * c - half : 8 * c;
    load8(row + i0, cc);
    load8(row + half + i0, ss);
#pragma unroll
    for (int i = 0; i < 8; ++i) {   // first half: a cos - b sin; second (x = b, y = a): b cos + a sin
      const float u = __fmul_rn(a[i], cc[i]), v = __fmul_rn(b[i], ss[i]);
      o[i] = second ? __fadd_rn(u, v) : __fsub_rn(u, v);
    }
  }
  return round8(o, dtype);
}

// Chunk c of the row at `row` (global memory), turned for position pos.
__device__ __forceinline__ uint4 turned_chunk(const RopeArgs& r, const uint16_t* row, int pos, int c, int dtype) {
  const uint4* w = reinterpret_cast<const uint4*>(row);
  const int p = partner(r, c);
  const uint4 x = w[c];
  return turn(r, pos, c, x, p == c ? x : w[p], dtype);
}

// Query row `row` (Hq heads of one token, at position pos) of q into q_out, by
// one warp; chunk pairs are read whole before either is written, so q_out may be q.
__device__ __forceinline__ void query_row(const RopeArgs& r, long long row, int pos, int dtype) {
  const int lane = threadIdx.x & 31;
  const uint4* src = reinterpret_cast<const uint4*>(r.q + row * r.Hq * kD);
  uint4* dst = reinterpret_cast<uint4*>(r.q_out + row * r.Hq * kD);
  const int n = r.Hq * 16;   // chunks of the row; a head's 16 sit in half a warp
  for (int base = 0; base < n; base += 32) {
    const int i = base + lane, c = i & 15;
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (i < n) x = src[i];
    const int from = (lane & 16) | partner(r, c);
    uint4 y;
    y.x = __shfl_sync(0xffffffffu, x.x, from);
    y.y = __shfl_sync(0xffffffffu, x.y, from);
    y.z = __shfl_sync(0xffffffffu, x.z, from);
    y.w = __shfl_sync(0xffffffffu, x.w, from);
    if (i < n) dst[i] = turn(r, pos, c, x, y, dtype);
  }
}

}  // namespace rope
}  // namespace s4kv
