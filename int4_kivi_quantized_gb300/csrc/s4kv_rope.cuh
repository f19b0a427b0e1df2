// Rotary position embedding of 16-bit rows, shared by the append kernels: an
// 8-channel chunk of a row turned by the angles of its position. Every product
// and sum is one binary32 rounding (no fused multiply-add) and the result is
// rounded once to the cache dtype, so the rows are those of a rotation done in
// 32-bit arithmetic before an ordinary append, bit for bit. Rotating apart from the
// append would read and write every key row once more (512 bytes beside the 770 that an
// INT8 append moves for a token and kv head); here it costs the angles, from L2.
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
  const float4 a = *reinterpret_cast<const float4*>(p), b = *(reinterpret_cast<const float4*>(p) + 1);
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
    const float4 cs = *reinterpret_cast<const float4*>(row + 4 * c);
    const float4 sn = *reinterpret_cast<const float4*>(row + half + 4 * c);
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

// What one lane turns of every head of a row: two chunks A and B and their angles.
// A head's 16 chunks are eight such units: the pairs of the rotation (u, u + half)
// and, past the rotated channels, plain neighbours; with interleaved pairs each
// chunk turns by itself (A by c, s 0..3, B by 4..7).
struct Unit {
  int A, B;
  bool turnA, turnB;
  float c[8], s[8];
};

__device__ __forceinline__ void unit_chunks(const RopeArgs& r, int u, Unit& x) {
  const int half = r.dim >> 4;
  if (r.interleaved) {
    x.A = u;
    x.B = u + 8;
    x.turnA = x.A < 2 * half;
    x.turnB = x.B < 2 * half;
  } else {
    x.turnA = x.turnB = u < half;
    x.A = u < half ? u : 2 * u;
    x.B = u < half ? u + half : 2 * u + 1;
  }
}

__device__ __forceinline__ void unit_angles(const RopeArgs& r, int pos, Unit& x) {
  const float* row = r.table + static_cast<long long>(pos) * r.dim;
  const int half = r.dim >> 1;
  if (!x.turnA) return;   // (B turns only where A does)
  const int a = r.interleaved ? 4 * x.A : 8 * x.A, b = r.interleaved ? (x.turnB ? 4 * x.B : a) : a + 4;
  const float4 c0 = *reinterpret_cast<const float4*>(row + a), c1 = *reinterpret_cast<const float4*>(row + b);
  const float4 s0 = *reinterpret_cast<const float4*>(row + half + a), s1 = *reinterpret_cast<const float4*>(row + half + b);
  x.c[0] = c0.x; x.c[1] = c0.y; x.c[2] = c0.z; x.c[3] = c0.w;
  x.c[4] = c1.x; x.c[5] = c1.y; x.c[6] = c1.z; x.c[7] = c1.w;
  x.s[0] = s0.x; x.s[1] = s0.y; x.s[2] = s0.z; x.s[3] = s0.w;
  x.s[4] = s1.x; x.s[5] = s1.y; x.s[6] = s1.z; x.s[7] = s1.w;
}

// The unit's chunks, turned in place.
template <int DT>
__device__ __forceinline__ void turn_unit(const RopeArgs& r, const Unit& x, uint4& A, uint4& B) {
  if (!x.turnA) return;
  float a[8], b[8], p[8], q[8];
  widen8(A, DT, a);
  widen8(B, DT, b);
  if (r.interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p[2 * i] = __fsub_rn(__fmul_rn(a[2 * i], x.c[i]), __fmul_rn(a[2 * i + 1], x.s[i]));
      p[2 * i + 1] = __fadd_rn(__fmul_rn(a[2 * i + 1], x.c[i]), __fmul_rn(a[2 * i], x.s[i]));
      q[2 * i] = __fsub_rn(__fmul_rn(b[2 * i], x.c[4 + i]), __fmul_rn(b[2 * i + 1], x.s[4 + i]));
      q[2 * i + 1] = __fadd_rn(__fmul_rn(b[2 * i + 1], x.c[4 + i]), __fmul_rn(b[2 * i], x.s[4 + i]));
    }
    A = round8(p, DT);
    if (x.turnB) B = round8(q, DT);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      p[i] = __fsub_rn(__fmul_rn(a[i], x.c[i]), __fmul_rn(b[i], x.s[i]));
      q[i] = __fadd_rn(__fmul_rn(b[i], x.c[i]), __fmul_rn(a[i], x.s[i]));
    }
    A = round8(p, DT);
    B = round8(q, DT);
  }
}

// Sequence that owns input row `row`: the last i with cu_new[i] <= row, 32 probes
// a round, by one warp.
__device__ __forceinline__ int sequence_of_row(const int* cu_new, int n, int row) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n;   // cu_new[lo] <= row, and hi is the end or past it
  while (hi - lo > 1) {
    const int gap = (hi - lo + 31) / 32, at = lo + gap * (lane + 1);
    const int k = __ffs(__ballot_sync(0xffffffffu, at >= hi || cu_new[at] > row)) - 1;
    lo += gap * k;
    hi = min(hi, lo + gap);
  }
  return lo;
}

// Queries of a call: items of one row and kQueryHeads heads, a warp each. All of an
// item's loads are in flight together (the rotation is nothing but bytes), its
// angles are read once for the item's heads, and every chunk is read before its
// pair is written, so q_out may be q.
constexpr int kQueryHeads = 16;
__host__ __device__ __forceinline__ long long query_items(const RopeArgs& r, int rows) {
  return r.q ? static_cast<long long>(rows) * ((r.Hq + kQueryHeads - 1) / kQueryHeads) : 0;
}
template <int DT>
__device__ __forceinline__ void query_item(const AppendArgs& a, long long item) {
  const RopeArgs& r = a.rope;
  const int lane = threadIdx.x & 31, blocks = (r.Hq + kQueryHeads - 1) / kQueryHeads;
  const int row = static_cast<int>(item / blocks), h0 = static_cast<int>(item - static_cast<long long>(row) * blocks) * kQueryHeads;
  Unit x;
  unit_chunks(r, lane & 7, x);
  const uint4* src = reinterpret_cast<const uint4*>(r.q + static_cast<long long>(row) * r.Hq * kD);
  uint4* dst = reinterpret_cast<uint4*>(r.q_out + static_cast<long long>(row) * r.Hq * kD);
  uint4 A[kQueryHeads / 4], B[kQueryHeads / 4];
#pragma unroll
  for (int i = 0; i < kQueryHeads / 4; ++i) {
    const int h = h0 + 4 * i + (lane >> 3);
    A[i] = B[i] = make_uint4(0u, 0u, 0u, 0u);
    if (h < r.Hq) {
      A[i] = src[16 * h + x.A];
      B[i] = src[16 * h + x.B];
    }
  }
  const int seq = sequence_of_row(a.cu_new, a.n, row);
  const int T0 = a.seq_lens_before[seq], c0 = a.cu_new[seq];
  if (T0 + a.cu_new[seq + 1] - c0 > r.max_pos) return;   // a token past the table: reported with the keys
  unit_angles(r, T0 + row - c0, x);
#pragma unroll
  for (int i = 0; i < kQueryHeads / 4; ++i) {
    const int h = h0 + 4 * i + (lane >> 3);
    turn_unit<DT>(r, x, A[i], B[i]);
    if (h < r.Hq) {
      dst[16 * h + x.A] = A[i];
      dst[16 * h + x.B] = B[i];
    }
  }
}

}  // namespace rope
}  // namespace s4kv
