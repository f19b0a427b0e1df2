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

#include "s4kv_restore.cuh"

#include <type_traits>

namespace s4kv {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
// (two or three of them, on the prompts above: INT8 16.6 / 19.4 us, 4-bit 17.8 / 27.2: at 80
// registers a lane keeps fewer loads in flight)
#ifndef S4KV_GATHER_CTAS
#define S4KV_GATHER_CTAS 2
#endif
constexpr int kCtas = S4KV_GATHER_CTAS;   // resident CTAs per SM the registers are budgeted for

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

// Rows of a dense tensor: token 0's at `at`, a token is `step` elements.
template <typename OUT>
struct Rows {
  OUT* at;
  int step;
  __device__ __forceinline__ void operator()(int token, int c, const float (&y)[8]) const {
    put8(at + static_cast<long long>(token) * step + 8 * c, y);
  }
};

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
        put_key_group<FMT>(rec, rec1, odd + lo, odd + hi, Rows<OUT>{dst - static_cast<long long>(odd) * step, step});
      }
      continue;
    }
    const Rows<OUT> rows_of{dst, step};
    const int held = min(max(quant - t0, lo), hi);   // tokens [lo, held) are in the record, [held, hi) in the ring
    if (held > lo) {
      if (values) put_values<FMT>(a.fp8_scale + a.H + h, rec, lo, held, rows_of);
      else if constexpr (kByte<FMT>) put_keys<FMT>(a.fp8_scale + h, rec, lo, held, rows_of);
    }
    if (FMT != 8 && hi > held) put_ring(ring, values ? vmod : kKMod, t0, held, hi, a.dtype, rows_of);
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
