// Batched restore (s4kv_gather): token ranges of many sequences out of the pages
// and rings into dense rows, for every page format. One pass over the records that
// the ranges need and one over the rows: bound by those bytes.
//
// Work item, one warp: one page of one kv head. The record is copied whole into
// shared memory with 16-byte loads (its bytes are in the order of the attention
// kernels' operands, not of rows); then lane (r, c) = (l / 16, l % 16) puts
// channels 8c .. 8c+7 of token 2 it + r together, so that every store instruction
// writes whole rows.
//
// Page slots: sequence i starts at slot cu_rows[i] / 16 + 2 i; a range of x rows
// touches at most x / 16 + 2 pages, so sequences do not overlap, and a slot finds
// its sequence by a search over cu_rows alone.
//
// Compiled without FMA contraction: a restored value is fmaf(code, scale, min)
// (KIVI) or code * scale (8-bit), rounded once more only to a 16-bit out_dtype.

#include "s4kv_common.cuh"

#include <cuda_fp8.h>

namespace s4kv {
namespace {

constexpr int kI8 = S4KV_BITS_INT8;
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
template <int FMT> constexpr bool kByte = FMT == 8 || FMT == kI8;
// Bytes of a record that are staged, in 16-byte units.
template <int FMT> constexpr int kUnits = FMT == kI8 ? Rec<kI8>::kCopy / 16 : Rec<FMT>::kBytes / 16;

__device__ __forceinline__ void put8(const GatherArgs& a, void* out, long long row, int h, int c, const float (&y)[8]) {
  const long long idx = (row * a.H + h) * kD + 8 * c;
  if (a.out_dtype == S4KV_F32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(out) + idx);
    p[0] = make_float4(y[0], y[1], y[2], y[3]);
    p[1] = make_float4(y[4], y[5], y[6], y[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (a.out_dtype == S4KV_BF16) {
        const __nv_bfloat162 x = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&x);
      } else {
        const __half2 x = __floats2half2_rn(y[2 * i], y[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&x);
      }
    }
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + idx) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// A ring row's chunk, widened exactly.
__device__ __forceinline__ void ring8(const uint16_t* row, int c, int dtype, float (&y)[8]) {
  const uint4 v = reinterpret_cast<const uint4*>(row)[c];
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[2 * i] = widen16(static_cast<uint16_t>(w[i] & 0xffff), dtype);
    y[2 * i + 1] = widen16(static_cast<uint16_t>(w[i] >> 16), dtype);
  }
}

__device__ __forceinline__ float e4m3(uint32_t byte) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(byte), __NV_E4M3)));
}
template <int FMT>
__device__ __forceinline__ float byte_value(uint32_t byte) {
  if constexpr (FMT == kI8) return static_cast<float>(static_cast<int>(byte) - 128);
  else return e4m3(byte);
}

// Key chunk c of token tau of the page staged at `rec`. KIVI: meta is the record
// (global memory) of the page of the pair that holds the chunk's scales.
template <int FMT>
__device__ __forceinline__ void key8(const char* rec, const char* meta, int tau, int c, float scale, float (&y)[8]) {
  const int at = tau & 7, hi = tau >> 3, L = 4 * at + (c >> 2);
  if constexpr (kByte<FMT>) {
    const uint4 v = *reinterpret_cast<const uint4*>(rec + (c & 3) * 512 + L * 16);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const uint32_t p = w[x] >> (16 * hi);
      y[2 * x] = __fmul_rn(byte_value<FMT>(p & 0xffu), scale);
      y[2 * x + 1] = __fmul_rn(byte_value<FMT>((p >> 8) & 0xffu), scale);
    }
  } else {
    using F = Rec<FMT>;
    const int u = (c >> 2) & 1, i = 2 * (c & 3);
#pragma unroll
    for (int half = 0; half < 2; ++half) {   // channels 8c + 4 half .. + 3: slice kk = 2 (c % 4) + half
      const float* m = reinterpret_cast<const float*>(meta + F::kKm + (2 * (i + half) + u) * 16);
      const float4 s4 = __ldg(reinterpret_cast<const float4*>(m)), m4 = __ldg(reinterpret_cast<const float4*>(m) + 16);
      uint32_t q;   // bytes c_0, c_2, c_1, c_3
      if constexpr (FMT == 4) {
        const int kk = i + half;
        q = *reinterpret_cast<const uint32_t*>(rec + F::kKc + (kk >> 2) * 512 + L * 16 + (kk & 3) * 4) >> (4 * hi);
        q &= 0x0f0f0f0fu;
      } else {
        q = *reinterpret_cast<const uint32_t*>(rec + F::kKc + L * 16 + (i >> 1) * 4) >> (2 * (2 * half + hi));
        q &= 0x03030303u;
      }
      y[4 * half + 0] = __fmaf_rn(static_cast<float>(q & 0xffu), s4.x, m4.x);
      y[4 * half + 1] = __fmaf_rn(static_cast<float>((q >> 16) & 0xffu), s4.y, m4.y);
      y[4 * half + 2] = __fmaf_rn(static_cast<float>((q >> 8) & 0xffu), s4.z, m4.z);
      y[4 * half + 3] = __fmaf_rn(static_cast<float>(q >> 24), s4.w, m4.w);
    }
  }
}

// Value chunk c of token tau of the page staged at `rec`.
template <int FMT>
__device__ __forceinline__ void value8(const char* rec, int tau, int c, float scale, float (&y)[8]) {
  const int b = (tau & 7) >> 1, r = tau & 1, w = tau >> 3;
  const uint8_t* p = reinterpret_cast<const uint8_t*>(rec);
  if constexpr (FMT == kI8) {   // channels 64 hi + 8a + m of lane 4a + b: words m / 2
    const int at = c & 7, hi = c >> 3;
#pragma unroll
    for (int m = 0; m < 8; ++m)
      y[m] = __fmul_rn(byte_value<FMT>(p[Rec<kI8>::kVc + (m >> 1) * 512 + (4 * at + b) * 16 + 8 * (m & 1) + 4 * w + 2 * hi + r]), scale);
  } else if constexpr (FMT == 8) {
    const int mt = c >> 1, up = c & 1;
#pragma unroll
    for (int at = 0; at < 8; ++at)
      y[at] = __fmul_rn(byte_value<FMT>(p[Rec<8>::kVc + (mt >> 1) * 512 + (4 * at + b) * 16 + 8 * (mt & 1) + 4 * w + 2 * up + r]), scale);
  } else {
    using F = Rec<FMT>;
    const int bt = w ? (r ? 3 : 1) : (r ? 2 : 0), e = r + 2 * w, k = c >> 2;
    const float s = *reinterpret_cast<const float*>(rec + F::kVm + ((2 * k) * 4 + b) * 16 + 4 * e);
    const float mn = *reinterpret_cast<const float*>(rec + F::kVm + ((2 * k + 1) * 4 + b) * 16 + 4 * e);
#pragma unroll
    for (int at = 0; at < 8; ++at) {
      uint32_t q;
      if constexpr (FMT == 4) {
        const int mt = c >> 1;
        q = (p[F::kVc + (mt >> 2) * 512 + (4 * at + b) * 16 + (mt & 3) * 4 + bt] >> (4 * (c & 1))) & 15u;
      } else {
        q = (p[F::kVc + (4 * at + b) * 16 + (c >> 2) * 4 + bt] >> (2 * (c & 3))) & 3u;
      }
      y[at] = __fmaf_rn(static_cast<float>(q), s, mn);
    }
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

template <int FMT>
__global__ void __launch_bounds__(kThreads) gather_kernel(GatherArgs a) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  char* rec = reinterpret_cast<char*>(smem_raw) + warp * (kUnits<FMT> * 16);
  {   // a malformed call: nothing is read or written
    int bad = a.cu_rows[0] != 0 || a.cu_rows[a.n] != a.num_rows;
    for (int i = threadIdx.x; i < a.n; i += kThreads) {
      const int f = a.first ? a.first[i] : 0;
      bad |= a.cu_rows[i + 1] < a.cu_rows[i] || f < 0 || f > (1 << 30) || a.cu_rows[i + 1] - a.cu_rows[i] > (1 << 30);
    }
    if (__syncthreads_or(bad)) {
      if (blockIdx.x == 0 && threadIdx.x == 0) report(a.status, S4KV_ERR_DEVICE, S4KV_DEV_BAD_CU, a.n);
      return;
    }
  }
  const long long total = (static_cast<long long>(a.num_rows) / kP + 2LL * a.n) * a.H;
  for (long long it = static_cast<long long>(blockIdx.x) * kWarps + warp; it < total; it += static_cast<long long>(gridDim.x) * kWarps) {
    const int s = static_cast<int>(it / a.H), h = static_cast<int>(it - static_cast<long long>(s) * a.H);
    const int i = sequence_of(a, s);
    const int f = a.first ? a.first[i] : 0, c0 = a.cu_rows[i], cnt = a.cu_rows[i + 1] - c0;
    const int page = f / kP + (s - slot_base(a, i));
    const int t0 = max(f, page * kP), t1 = min(f + cnt, page * kP + kP);
    const int T = a.seq_lens[i], slot = a.slot_ids ? a.slot_ids[i] : i;
    if (cnt == 0 || t0 >= t1) continue;
    int bad = 0, arg = i;
    if (slot < 0 || slot >= a.max_slots) {
      bad = S4KV_DEV_BAD_SLOT;
      arg = slot;
    } else if (T < 0 || a.lens[slot * a.H + h] != T) {
      bad = S4KV_DEV_BAD_LENGTH;
    } else if (f + cnt > T) {
      bad = S4KV_DEV_BAD_POSITION;
    } else if (static_cast<long long>(a.bt_stride) * kP < f + cnt) {
      bad = S4KV_DEV_BAD_TABLE;
    }
    if (bad) {
      if (lane == 0) report(a.status, S4KV_ERR_DEVICE, bad, arg);
      continue;
    }
    // first token of the key and of the value residual
    const int Tk = FMT == 8 ? T : FMT == kI8 ? T / kP * kP : T & ~(kG - 1);
    const int Tv = FMT == 8 ? T : FMT == kI8 ? Tk : max(0, T - a.R);
    const int* bt = a.block_table + static_cast<long long>(i) * a.bt_stride;
    const char* meta[2] = {nullptr, nullptr};
    float ks = 1.0f, vs = 1.0f;
    const bool paged = t0 < max(Tk, Tv);
    if (paged) {
      int pp = bt[page], p0 = pp, p1 = pp;
      if constexpr (!kByte<FMT>) {
        if (t0 < Tk) {   // the key metadata of a group spans its two pages
          p0 = bt[page & ~1];
          p1 = bt[page | 1];
        }
      }
      const bool out = pp < 0 || pp >= a.num_pages || p0 < 0 || p0 >= a.num_pages || p1 < 0 || p1 >= a.num_pages;
      if (out) {
        if (lane == 0) report(a.status, S4KV_ERR_DEVICE, S4KV_DEV_BAD_PAGE, pp < 0 || pp >= a.num_pages ? pp : p0 < 0 || p0 >= a.num_pages ? p0 : p1);
        continue;
      }
      const char* src = a.pages + (static_cast<long long>(pp) * a.H + h) * Rec<FMT>::kBytes;
      meta[0] = a.pages + (static_cast<long long>(p0) * a.H + h) * Rec<FMT>::kBytes;
      meta[1] = a.pages + (static_cast<long long>(p1) * a.H + h) * Rec<FMT>::kBytes;
      __syncwarp();   // the previous item's readers are done
#pragma unroll
      for (int u = 0; u < kUnits<FMT>; u += 32)
        if (u + lane < kUnits<FMT>)
          reinterpret_cast<uint4*>(rec)[u + lane] = __ldg(reinterpret_cast<const uint4*>(src) + u + lane);
      __syncwarp();
      if constexpr (FMT == kI8) {
        ks = *reinterpret_cast<const float*>(rec + Rec<kI8>::kKs);
        vs = *reinterpret_cast<const float*>(rec + Rec<kI8>::kVs);
      } else if constexpr (FMT == 8) {
        ks = a.fp8_scale[h];
        vs = a.fp8_scale[a.H + h];
      }
    }
    const uint16_t* kring = reinterpret_cast<const uint16_t*>(a.kring) + slot * a.kring_slot + h * a.kring_head;
    const uint16_t* vring = reinterpret_cast<const uint16_t*>(a.vring) + slot * a.vring_slot + h * a.vring_head;
    constexpr int kKMod = FMT == kI8 ? kP : kG;
    const int vmod = FMT == kI8 ? kP : a.R;
    const int c = lane & 15;
#pragma unroll 2
    for (int x = 0; x < 8; ++x) {
      const int tau = 2 * x + (lane >> 4), t = page * kP + tau;
      if (t < t0 || t >= t1) continue;
      const long long row = c0 + (t - f);
      float y[8];
      if (FMT == 8 || t < Tk) key8<FMT>(rec, meta[c >> 3], tau, c, ks, y);
      else ring8(kring + static_cast<long long>(t % kKMod) * kD, c, a.dtype, y);
      put8(a, a.out_k, row, h, c, y);
      if (FMT == 8 || t < Tv) value8<FMT>(rec, tau, c, vs, y);
      else ring8(vring + static_cast<long long>(t % vmod) * kD, c, a.dtype, y);
      put8(a, a.out_v, row, h, c, y);
    }
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

template <int FMT>
cudaError_t run(const GatherArgs& a, int num_sms, cudaStream_t st) {
  const cudaError_t c = prefer_max_shared(reinterpret_cast<const void*>(gather_kernel<FMT>));
  if (c != cudaSuccess) return c;
  const long long items = (static_cast<long long>(a.num_rows) / kP + 2LL * a.n) * a.H;
  const long long want = (items + kWarps - 1) / kWarps, cap = static_cast<long long>(num_sms) * 6;
  gather_kernel<FMT><<<static_cast<unsigned>(want < cap ? want : cap), kThreads, kWarps * kUnits<FMT> * 16, st>>>(a);
  return cudaGetLastError();
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
