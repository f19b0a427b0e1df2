// Prompt attention (s4kv_prompt_attention): the chunks of new tokens of every sequence, of any
// lengths, over their cached tokens, with a score form. tcgen05 with accumulators in tensor
// memory, warp-specialized.
//
// A row is one query token and one of the g query heads of a kv head; a CTA holds 256 rows of a
// sequence and kv head as two tiles of 128 and walks the kv tiles (128 tokens) that one of its
// rows sees. For each tile of rows
//     S = Q K^T (128 x 128 x 128),  P = exp2(score form(S) - m),  O += P V (128 x 128 x 128)
// with S and O in tensor memory; P, in f16, takes S's place there and is the A operand of
// P V. One thread a row: its 128 scores come in registers, so maxima and sums need no
// shuffle, and a rescale of O (when a maximum rises by more than kLazyP above the last one) is the row's own.
//
// Warps 0 .. 3 and 4 .. 7 are the rows of the two tiles, warp 8 fetches (a ring of five 32 KB
// buffers, keys and values in turn, one bulk copy each), warp 9 issues the MMAs: P V and the next
// Q K^T of one tile while the other tile's rows are at their exponentials. The tensor
// cores execute one thread's MMAs in the order of issue, so that the next scores overwrite P
// only when P V has read it.
//
// Few rows behind a long cache: the kv tiles of a CTA are split over `splits` CTAs, whose
// outputs a third launch combines.
//
// Two tiles of rows share a kv tile's fetch: 64 KB out of L2 for 256 x 128 scores keep ahead of the MMAs,
// where tiles of 128 rows alone would ask for twice that.
//
// Measured (one launch with its tiles and combine, a captured graph): 2048 tokens behind 32768, 28 query
// heads, 4 kv heads 626 us, 1490 TFLOP/s of the visible pairs (78% of a library matrix product's rate),
// with a cap of 30 and scores near zero 823, with scores beyond it 1390, with slopes 807, with both
// 1115. A prompt of 2048, 32 heads 44 to 46 (780 to 750). Eight chunks of 512 behind 2048 to 8192, sloped 351. What
// bounds it:
//  * the loop: 2811 cycles a kv tile, of which the four MMAs take 2052 (513 each, read out of shared
//    memory or with P out of tensor memory alike); the rest is P's way to tensor memory and the hand-over.
//    With a cap the rows' warps bind: 4170 cycles, a minimum more over the scores, and for two of them a
//    product and three multiply-adds (packed) beside the exponentials'.
//  * a CTA's start and end, about 15000 cycles: the sequence found (1400) and checked, queries fetched
//    and turned into operands (bf16 1500: its powers of two), first scores (2700), output (5800).
//    That is what a prompt of 2048 spends beside 16 kv tiles at most, hence tiles by falling length, and
//    the start runs beside the tiles' launch where that leaves SMs free (a prompt of 512 19.6 -> 16.8 us).
// Tried and left out: exponentials by polynomials on the FMA pipe, two threads a row, two MMA warps, P
// handed over in halves, barrier tests ahead of the waits: slower or level. Barriers shared by the
// two row tiles 2% faster, with an end that cannot be drained in bounded time.

#include "s4kv_prompt.cuh"
#include "s4kv_tcgen05.cuh"

#include <mutex>
#include <type_traits>

namespace s4kv {
namespace {

constexpr int kRowWarps = 8, kLoadWarp = 8, kMmaWarp = 9;
constexpr int kThreads = 384;        // (two more warps make a warpgroup of the last four)
// Registers: 168 a thread at launch, 224 for the rows' two warpgroups and 56 for the third (208 and 88: the capped
// rows spill more, 32k 831 us against 820).
constexpr int kRegsRow = 224, kRegsRest = 56;
static_assert(2 * kRegsRow + kRegsRest <= 3 * 168, "the shares are what the launch holds");
constexpr int kBufs = 5;
// A row's reference stands kRoom below the largest score so far and rises when one passes it by more than
// kRoom + kLazyP: P up to 2^15 in f16 before its sum divides it, so that rescales are rare, and what lies 2^-21
// below the largest keeps its 11 bits, what lies 2^-32 below it one.
constexpr float kLazyP = 8.0f, kRoom = 7.0f;
constexpr int kQBytes = 128 * kD * 2;
constexpr int kSmemBytes = 2 * kQBytes + kBufs * kTileBytes + 1024;
// tensor memory columns: S (and P) of tile s at 128 s, O at 256 + 128 s
constexpr uint32_t kTmemCols = 512;

// The MMAs, by descriptors in two words: the upper one is the same for every operand (rows of 128
// swizzled bytes, eight of them 1024 bytes), the lower one a start address / 16 plus the leading
// byte offset / 16 at bit 16, so that the next K-step is an addition (umma_desc composes a
// descriptor's fields, ten instructions between two MMAs).
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (kSw128 << 29);
constexpr uint32_t kDescK = 1u << 16;                     // K-major: unused
constexpr uint32_t kDescMn = (16384u >> 4) << 16;         // MN-major: from one 64 channels to the next
__device__ __forceinline__ void umma_ss(uint32_t d_tmem, uint32_t a_low, uint32_t b_low, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.u32 p, %5, 0;\n\tmov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_low), "r"(b_low), "r"(kDescHigh), "r"(idesc), "r"(acc ? 1u : 0u)
      : "memory");
}
// A in tensor memory: f16 pairs, a row a lane.
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_low, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.u32 p, %5, 0;\n\tmov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_low), "r"(kDescHigh), "r"(idesc), "r"(acc ? 1u : 0u)
      : "memory");
}
// One lane of a converged warp, the same every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
constexpr uint32_t kIdescQK = umma_idesc(128, 128);
constexpr uint32_t kIdescPV = umma_idesc(128, 128) | (1u << 16);   // B is MN-major

// mbar_try_wait that lets the thread sleep inside for up to `ns`: warps that poll take the shared
// memory's bandwidth from the operands (a 32k prompt: 750 us, polling 823).
__device__ __forceinline__ bool mbar_try_wait_for(uint64_t* bar, uint32_t parity, uint32_t ns) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(ns)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

struct PromptSmem {
  alignas(8) uint64_t full[kBufs], empty[kBufs];
  uint64_t sfull[2], pfull[2], odone[2], drain;
  float up[kQRows];           // a row's scores come out this much too small (its query's power of two)
  int lo, hi, abort;
  uint32_t tmem;
};

__device__ __forceinline__ float* part_rows(const PromptArgs& a, long long item) { return a.part + item * (kQRows * kD); }
__device__ __forceinline__ float* part_ml(const PromptArgs& a, long long item) {
  return a.part + static_cast<long long>(a.q_tiles) * a.H * a.splits * (kQRows * kD) + item * (2 * kQRows);
}

// The larger (smaller) of three numbers: one instruction.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
  float y;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// One row's scores of a kv tile, from S to log2 units.
struct RowScore {
  float mul;       // no cap: S to log2 units. cap: S to x / cap. A normal number
  float cap2;      // cap log2(e)
  float slope2;    // slope log2(e)
};

// The cap of a score near zero against it (s4kv_score.cuh), from S to log2 units: S Q(S^2) with Q's
// coefficients at hand per row. The last of them has the seventh power of x / (cap S): where it or the
// first is no normal number (large and tiny caps, rows of small queries), u = S mul comes first.
struct NearCap {
  float c[kNearCoefs];
  __device__ __forceinline__ NearCap(float lin, float mul) {   // lin: S to x in log2 units
    float by = lin;
#pragma unroll
    for (int k = 0; k < kNearCoefs; ++k, by *= mul * mul) c[k] = near_coef(k) * by;
  }
  __device__ __forceinline__ static bool normal(float x) { return fabsf(x) > 1e-36f && fabsf(x) < 1e36f; }
  __device__ __forceinline__ bool folds() const { return normal(c[0]) && normal(c[kNearCoefs - 1]); }   // (those between lie between)
  __device__ __forceinline__ float2 inner(float2 s) const {   // Q(S^2)
    const float2 w = __fmul2_rn(s, s);
    float2 p = __ffma2_rn(w, make_float2(c[3], c[3]), make_float2(c[2], c[2]));
    p = __ffma2_rn(p, w, make_float2(c[1], c[1]));
    return __ffma2_rn(p, w, make_float2(c[0], c[0]));
  }
  __device__ __forceinline__ float operator()(float s) const { return s * inner(make_float2(s, s)).x; }
};

// x from S to capped scores in log2 units, near zero (by the folded coefficients or not) or anywhere.
__device__ __forceinline__ void through_cap(float (&x)[128], const RowScore& f, const NearCap& near, bool near_zero, bool folded, float lin) {
  if (near_zero && folded) {
#pragma unroll
    for (int i = 0; i < 128; i += 2) {
      const float2 s = make_float2(x[i], x[i + 1]), y = __fmul2_rn(s, near.inner(s));
      x[i] = y.x;
      x[i + 1] = y.y;
    }
  } else if (near_zero) {
#pragma unroll
    for (int i = 0; i < 128; i += 2) {
      const float2 s = make_float2(x[i], x[i + 1]), u = __fmul2_rn(s, make_float2(f.mul, f.mul)), w = __fmul2_rn(u, u);
      float2 p = make_float2(near_coef(3), near_coef(3));
#pragma unroll
      for (int k = kNearCoefs - 2; k >= 0; --k) p = __ffma2_rn(p, w, make_float2(near_coef(k), near_coef(k)));
      const float2 y = __fmul2_rn(__fmul2_rn(s, make_float2(lin, lin)), p);
      x[i] = y.x;
      x[i + 1] = y.y;
    }
  } else {
    const float by = f.mul * 2.8853900817779268f;   // 2 log2(e)
#pragma unroll
    for (int i = 0; i < 128; ++i) x[i] = far_cap(x[i], by, f.cap2);
  }
}

template <bool CAP, bool SLOPE>
__global__ void __launch_bounds__(kThreads, 1) prompt_kernel(PromptArgs a) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  __shared__ PromptSmem sm;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  char* q_tiles = reinterpret_cast<char*>(smem_raw) + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  char* ring = q_tiles + 2 * kQBytes;
  if (tid == 0) {
    sm.abort = 0;
    sm.lo = 0x7fffffff;
    sm.hi = -1;
  }
  __syncthreads();
  // What the caller's work made is there: the tiles' launch has waited for it, and lets this one start then. This
  // kernel reads it past the first cache, and waits for the tiles themselves further down (on every path, so
  // that its end is theirs).
  Place pl;
  // the last tiles of a sequence, whose rows see the most, start first, of every kv head
  const int q_tile = static_cast<int>((gridDim.x - 1 - blockIdx.x) / a.H), h = static_cast<int>(blockIdx.x % a.H);
  const int where = find_tile<kThreads, true>(a, q_tile, pl);
  // (no branch: a path of its own would cost the loop registers)
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.s32 p, %0, 0;\n\t@p griddepcontrol.wait;\n\t}" ::"r"(where) : "memory");
  if (where != kFound) return;
  const int z = blockIdx.y, b = pl.b, g = a.g, cu0 = pl.cu0, m = pl.m, T = pl.T;
  const int row0 = pl.tile * kQRows;
  const int rows = static_cast<int>(min(static_cast<long long>(kQRows), static_cast<long long>(m) * g - row0));
  const int tiles = rows > 128 ? 2 : 1;
  // a row's token of the chunk; its row of q and out
  const int tok0 = row0 / g, rem0 = row0 - tok0 * g, by_g = 65536 / g + 1;   // x / g = x by_g >> 16 for x < 264, g <= 8
  auto token_of = [&](int r) { return tok0 + ((rem0 + r) * by_g >> 16); };
  auto out_row = [&](int r) -> long long {
    const int i = token_of(r);
    return (static_cast<long long>(cu0) + i) * a.Hq + h * g + (row0 + r - i * g);
  };
  if (tid == 0) {
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm.sfull[s], 1);
      mbar_init(&sm.pfull[s], 4);
      mbar_init(&sm.odone[s], 1);
    }
    mbar_init(&sm.drain, 1);
  }
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  uint4 v[16];   // the queries on their way: a warp's 32 rows, two at a time
  if (warp < kRowWarps) {
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const int r = 32 * warp + 2 * k + (lane >> 4);
      v[k] = r < rows ? __ldcg(reinterpret_cast<const uint4*>(a.q + out_row(r) * kD) + (lane & 15)) : make_uint4(0u, 0u, 0u, 0u);
    }
  }
  const int slot = a.slot_ids ? __ldcg(a.slot_ids + b) : b;
  int arg;
  const int why = refused(a, pl, slot, h, arg);
  if (why && tid == 0) report(a.status, S4KV_ERR_DEVICE, why, arg);

  // ---- what each row sees; the queries as f16 operands ----
  Span sp{0, 0x7fffffff};   // (rows past the last one: everything, so that they ask for no masks)
  int pos = 0;
  if (warp < kRowWarps && !why) {
    if (tid < rows) {
      const int i = token_of(tid);
      pos = T - m + i;
      sp = span_of<true>(a.form, pos, T, static_cast<long long>(cu0) + i, b);
    }
    const bool range = tid < rows && sp.lo <= sp.hi;
    const int lo = __reduce_min_sync(0xffffffffu, range ? sp.lo : 0x7fffffff);
    const int hi = __reduce_max_sync(0xffffffffu, tid < rows ? sp.hi : -1);
    if (lane == 0) {
      atomicMin(&sm.lo, lo);
      atomicMax(&sm.hi, hi);
    }
    // f16 operands, swizzled. bf16 has the wider range: a row is taken at the power of two that brings its
    // largest element to 2^3 .. 2^4: exact, elements down to 2^-17, 2^-20 of the largest, keep every bit, smaller
    // ones are off by 2^-25 at most (2^-28 of the largest), and powers of what then scales the scores stay
    // normal numbers where they can.
    const int c = lane & 15;
    float up = 1.0f;   // of row lane % 16 of this half warp's
    if (a.dtype == S4KV_BF16) {
      uint32_t top[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        constexpr uint32_t kAbs = 0x7fff7fffu;
        const uint32_t t = __vimax3_u16x2(__vimax3_u16x2(v[k].x & kAbs, v[k].y & kAbs, v[k].z & kAbs), v[k].w & kAbs, 0u);
        top[k] = max(t & 0xffffu, t >> 16);
      }
      // over the 16 lanes: each step halves the rows that a lane goes on with
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) {
        const bool upper = lane & o;
#pragma unroll
        for (int k = 0; k < o; ++k) {
          const uint32_t keep = upper ? top[k + o] : top[k], send = upper ? top[k] : top[k + o];
          top[k] = max(keep, __shfl_xor_sync(0xffffffffu, send, o));
        }
      }
      const int e = static_cast<int>(top[0] >> 7), pw = top[0] == 0 || e == 255 ? 0 : min(3 + 127 - e, 126);
      up = power_of_two(pw);
      sm.up[32 * warp + 2 * c + (lane >> 4)] = power_of_two(-pw);
    } else {
      sm.up[tid] = 1.0f;
    }
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const int r = 32 * warp + 2 * k + (lane >> 4);
      uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
      if (a.dtype == S4KV_BF16) {
        const float by = __shfl_sync(0xffffffffu, up, (lane & 16) | k);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = pack_f16x2(__uint_as_float(w[i] << 16) * by, __uint_as_float(w[i] & 0xffff0000u) * by);
      }
      *reinterpret_cast<uint4*>(q_tiles + (r >> 7) * kQBytes + sw128_off(r & 127, 8 * c, 128)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    fence_proxy_async();
  }
  if (warp == kLoadWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm.tmem)), "n"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  stream_wait();   // (no early start for what comes behind: its CTAs would crowd the SMs that end first)
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  // kv tiles that some row sees: the sinks' [0, sa), then [jb, je) (restored all: the sequence's range holds them)
  const int last = sm.hi;
  const int sa = why ? 0 : (min(a.form.sinks, last + 1) + kKvTile - 1) / kKvTile;
  const int jb = max(sa, sm.lo == 0x7fffffff ? sa : sm.lo / kKvTile), je = why || sm.lo == 0x7fffffff ? jb : last / kKvTile + 1;
  const int all = sa + max(0, je - jb);
  const int i0 = static_cast<int>(static_cast<long long>(all) * z / a.splits);
  const int cnt = static_cast<int>(static_cast<long long>(all) * (z + 1) / a.splits) - i0;
  auto kv_of = [&](int i) { return i0 + i < sa ? i0 + i : jb + (i0 + i - sa); };
  const KvRange kept = kv_range(a, m, max(T, 1));
  auto tile_at = [&](int i) { return (static_cast<long long>(pl.kv0) + kept.at(kv_of(i))) * a.H + h; };

  volatile int* flag = &sm.abort;
  // Bounded: false, and the flag that ends every role's loop raised, when it runs out.
  auto wait = [&](uint64_t* bar, int parity) -> bool {
    unsigned long long t0 = 0;
    for (unsigned it = 1; a.wait_ns > 0; ++it) {
      if (mbar_try_wait_for(bar, parity, 20000u)) return true;
      if (*flag) return false;
      if ((it & 15u) == 0) {   // (reading the timer takes longer than most waits)
        const unsigned long long now = global_ns();
        if (t0 == 0) t0 = now;
        if (static_cast<long long>(now - t0) > a.wait_ns) break;
      }
    }
    *flag = 1;
    return false;
  };

  if (warp >= kRowWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
    if (warp == kLoadWarp) {
      if (lane == 0) {
        int sent = 0;
        bool ok = true;
        for (int it = 0; it < 2 * cnt; ++it) {
          const int s = it % kBufs;
          if (it >= kBufs) ok = wait(&sm.empty[s], (it / kBufs - 1) & 1);
          if (!ok) break;
          mbar_expect_tx(&sm.full[s], kTileBytes);
          asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                           smem_u32(ring + s * kTileBytes)),
                       "l"(a.tiles + (2 * tile_at(it >> 1) + (it & 1)) * kTileBytes), "r"(kTileBytes), "r"(smem_u32(&sm.full[s]))
                       : "memory");
          sent = it + 1;
        }
        // every copy has landed before the CTA ends
        for (int it = max(0, sent - kBufs); it < sent; ++it)
          if (!mbar_wait(&sm.full[it % kBufs], (it / kBufs) & 1, kDrainNs)) *flag = 1;
      }
      __syncwarp();
    } else if (warp == kMmaWarp) {
      // The whole warp walks the loop, so that addresses and counters are uniform; one lane issues.
      const uint32_t q_low = (smem_u32(q_tiles) >> 4) | kDescK, k_low = (smem_u32(ring) >> 4) | kDescK, v_low = (smem_u32(ring) >> 4) | kDescMn;
      auto qk = [&](int s, int slot) {
        const uint32_t b = k_low + slot * (kTileBytes >> 4), q = q_low + s * (kQBytes >> 4);
#pragma unroll
        for (int j = 0; j < 8; ++j) {   // 16 channels: 32 bytes, or on to the other 64 channels
          const uint32_t at = (j >> 2) * (16384 >> 4) + (j & 3) * (32 >> 4);
          umma_ss(tmem + 128 * s, q + at, b + at, kIdescQK, j > 0);
        }
        umma_commit(&sm.sfull[s]);
      };
      auto pv = [&](int s, int slot, bool acc) {
        const uint32_t b = v_low + slot * (kTileBytes >> 4);
#pragma unroll
        for (int j = 0; j < 8; ++j)   // 16 tokens: 8 columns of P, 16 rows of 128 bytes
          umma_ts(tmem + 256 + 128 * s, tmem + 128 * s + 8 * j, b + j * (2048 >> 4), kIdescPV, acc || j > 0);
        umma_commit(&sm.odone[s]);
      };
      auto all_wait = [&](uint64_t* bar, int parity) -> bool { return __all_sync(0xffffffffu, wait(bar, parity)); };
      if (cnt > 0) {
        bool ok = all_wait(&sm.full[0], 0);
        if (ok) {
          tc_fence_after();
          if (elect_one()) {
            qk(0, 0);
            if (tiles == 2) qk(1, 0);
            umma_commit(&sm.empty[0]);
          }
          __syncwarp();
        }
        int slot = 0, round = 0;   // of the ring; the parity of its rounds
        auto step = [&]() {
          slot = slot + 1 == kBufs ? 0 : slot + 1;
          round ^= slot == 0;
        };
        for (int i = 0; ok && i < cnt; ++i) {
          const bool more = i + 1 < cnt;
          // (the waits for copies, long there, go where the other tile's MMAs are still running)
          step();
          ok = all_wait(&sm.full[slot], round);              // values of tile i
          const int vslot = slot;
          step();
          if (ok && more) ok = all_wait(&sm.full[slot], round);   // keys of tile i + 1
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            if (s >= tiles) break;
            ok = ok && all_wait(&sm.pfull[s], i & 1);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
              pv(s, vslot, i > 0);
              if (s == tiles - 1) umma_commit(&sm.empty[vslot]);
              if (more) {
                qk(s, slot);
                if (s == tiles - 1) umma_commit(&sm.empty[slot]);
              }
            }
            __syncwarp();
          }
        }
        // no MMA is in flight when the CTA ends
        if (elect_one()) umma_commit(&sm.drain);
        __syncwarp();
        if (!mbar_wait(&sm.drain, 0, kDrainNs)) *flag = 1;
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsRow));
    if ((warp >> 2) < tiles) {
      const int s = warp >> 2;
      const uint32_t t_row = static_cast<uint32_t>(32 * (warp & 3)) << 16;
      const uint32_t s_at = tmem + 128 * s + t_row, o_at = tmem + 256 + 128 * s + t_row;
      constexpr float kLog2e = 1.4426950408889634f;
      RowScore f;
      const float key_scale = a.bits == 8 ? a.fp8_scale[h] : 1.0f;   // (FP8: the tiles hold codes)
      const float scale = a.sm_scale * sm.up[tid] * key_scale, lin = scale * kLog2e;
      f.mul = fminf(fmaxf(CAP ? scale / a.form.cap : lin, 0x1p-126f), 0x1p127f);   // (zero times it is zero, -inf -inf)
      f.cap2 = CAP ? a.form.cap * kLog2e : 0.0f;
      f.slope2 = SLOPE ? a.form.slopes[h * g + (row0 + tid) % g] * kLog2e : 0.0f;
      if (CAP) sm.up[tid] = lin;   // (this thread's own; seldom asked for)
      const NearCap near(lin, f.mul);
      const bool folded = CAP && __all_sync(0xffffffffu, near.folds());
      float mx = -INFINITY, l = 0.0f;
      bool ok = true;
      auto wild_of = [&](int i) { return *reinterpret_cast<const uint4*>(a.bad + 4 * tile_at(i)); };
      uint4 next = cnt > 0 ? wild_of(0) : make_uint4(0u, 0u, 0u, 0u);
      for (int i = 0; i < cnt; ++i) {
        const int t0 = kv_of(i) * kKvTile;
        const uint4 wild = next;
        if (i + 1 < cnt) next = wild_of(i + 1);
        const bool row_sees = t0 + kKvTile - 1 <= sp.hi && (t0 >= sp.lo || t0 + kKvTile <= a.form.sinks);
        const bool clean = (wild.x | wild.y | wild.z | wild.w) == 0;
        const bool all_see = CAP && __all_sync(0xffffffffu, row_sees);   // (caps alone ask for it: two votes cost 1% of a sloped prompt)
        const bool whole = CAP ? all_see && clean : __all_sync(0xffffffffu, row_sees && clean);
        ok = __all_sync(0xffffffffu, wait(&sm.sfull[s], i & 1));
        if (!ok) break;
        tc_fence_after();
        float x[128];
        {
          uint32_t(&r)[4][32] = reinterpret_cast<uint32_t(&)[4][32]>(x);
#pragma unroll
          for (int k = 0; k < 4; ++k) tmem_ld32(s_at + 32 * k, r[k]);
          tmem_wait_ld();
        }
        auto largest = [&]() {
          float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int j = 0; j < 128; j += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e) t4[e] = max3(t4[e], x[j + 2 * e], x[j + 2 * e + 1]);
          return fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
        };
        // bits of the row's visible tokens of 32
        auto below = [](int n) -> uint32_t { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; };
        auto seen_of = [&](int k) -> uint32_t {
          const int t = t0 + 32 * k;
          // (hi may be the largest int)
          return below(sp.hi - t >= 31 ? 32 : sp.hi - t + 1) & (~below(sp.lo - t) | below(a.form.sinks - t));
        };
        // What is left to do to x at the exponentials: x in + at gives log2 units (`in` > 0), so that S
        // stays S as long as it can; or (raw) the cap near zero, where every score of the warp is seen
        // and so near it.
        bool raw = CAP && !SLOPE && whole;
        float in = f.mul, at = 0.0f, far = 0.0f, top = 0.0f;
        if constexpr (CAP) {
          if (!all_see) {   // what a row does not see has no say in how its scores are capped
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t seen = seen_of(k);
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                float& y = x[32 * k + j];
                y = (seen >> j) & 1u ? y : 0.0f;
              }
            }
          }
          float t4[4] = {INFINITY, INFINITY, INFINITY, INFINITY};
#pragma unroll
          for (int j = 0; j < 128; j += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e) t4[e] = min3(t4[e], x[j + 2 * e], x[j + 2 * e + 1]);
          const float least = fminf(fminf(t4[0], t4[1]), fminf(t4[2], t4[3]));
          top = largest();
          far = fmaxf(top, -least);
          // Rows that see the same tokens decide together, others alone. (With slopes the first have a call of
          // their own, without a divergent branch: 1118 us against 1162 for 2048 tokens behind 32768.)
          const bool row_near = far * f.mul <= kNearCap, all_near = __all_sync(0xffffffffu, row_near);
          raw = raw && all_near && folded;
          if (!raw) {
            if (SLOPE && all_see) through_cap(x, f, near, all_near, folded, sm.up[tid]);
            else through_cap(x, f, near, all_see ? all_near : row_near, folded, sm.up[tid]);
            __syncwarp();
          }
          in = 1.0f;
        }
        if constexpr (SLOPE) {
          const float rel = static_cast<float>(pos - t0);
          const float by = CAP ? f.slope2 : f.slope2 / f.mul;   // in x's units
          if (__all_sync(0xffffffffu, rel >= 127.0f && fabsf(by) < 1e30f)) {   // every token before the query: the distance falls along the row
            at = -f.slope2 * rel;
#pragma unroll
            for (int j = 0; j < 128; ++j) x[j] = fmaf(by, static_cast<float>(j), x[j]);
          } else {
#pragma unroll
            for (int j = 0; j < 128; ++j) x[j] = fmaf(-f.slope2, fabsf(static_cast<float>(j) - rel), x[j] * in);
            in = 1.0f;
          }
        }
        if (!whole) {
          const uint32_t wilds[4] = {wild.x, wild.y, wild.z, wild.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t seen = seen_of(k);
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              float& y = x[32 * k + j];
              y = (seen >> j) & 1u ? y : -INFINITY;
            }
            const uint32_t poison = seen & wilds[k];
            if (poison)
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if ((poison >> j) & 1u) x[32 * k + j] = __int_as_float(0x7fffffff);
          }
        }
        if (raw) top = near(top);
        else top = fmaf(largest(), in, at);
        if (__any_sync(0xffffffffu, top > mx + (kRoom + kLazyP))) {
          const float mn = top > mx + (kRoom + kLazyP) ? top - kRoom : mx;
          const float by = mx == mn ? 1.0f : mx == -INFINITY ? 0.0f : exp2_fast(mx - mn);   // (nothing so far: l and O are zeros)
          if (i > 0) {
            ok = __all_sync(0xffffffffu, wait(&sm.odone[s], (i - 1) & 1));
            if (!ok) break;
            tc_fence_after();
            l *= by;
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {
              uint32_t o[32];
              tmem_ld32(o_at + 32 * k, o);
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * by);
              tmem_st32(o_at + 32 * k, o);
            }
            tmem_wait_st();
          }
          mx = mn;
        }
        const float base = mx == -INFINITY ? 0.0f : mx;   // (a row that has seen nothing: every p is zero)
        float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
        auto exponentials = [&](auto capped) {
          const float2 in2 = make_float2(in, in), off2 = make_float2(at - base, at - base);
          auto pair = [&](int j) -> uint32_t {
            float2 y = make_float2(x[2 * j], x[2 * j + 1]);
            y = __ffma2_rn(y, decltype(capped)::value ? near.inner(y) : in2, off2);
            y = make_float2(exp2_fast(y.x), exp2_fast(y.y));
            sum[j & 1] = __fadd2_rn(sum[j & 1], y);
            return pack_f16x2(y.x, y.y);
          };
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t w[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) w[j] = pair(32 * k + j);
            tmem_st32(s_at + 32 * k, w);
          }
        };
        if (CAP && !SLOPE && raw) exponentials(std::true_type{});
        else exponentials(std::false_type{});
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.pfull[s]);
      }
      // ---- the rows' output, or their part of it ----
      if (ok && cnt > 0) ok = __all_sync(0xffffffffu, wait(&sm.odone[s], (cnt - 1) & 1));
      tc_fence_after();
      const bool some = ok && cnt > 0;
      const long long item = (static_cast<long long>(q_tile) * a.H + h) * a.splits + z;
      const float value_scale = a.bits == 8 ? a.fp8_scale[a.H + h] : 1.0f;
      const float inv = (a.splits > 1 ? 1.0f : l > 0.0f ? 1.0f / l : l == l ? 0.0f : l) * value_scale;
      // Through the queries' place in shared memory (nothing reads them any more), so that a warp writes whole
      // rows: 16 chunks of 16 bytes, chunk c of row r at c xor (r mod 16). 32 bits: in two goes.
      char* stage = q_tiles + s * kQBytes + (warp & 3) * 32 * 256;
      const bool f32 = a.splits > 1 || a.out_dtype == S4KV_F32;
      char* to = reinterpret_cast<char*>(a.splits > 1 ? part_rows(a, item) : a.out);
#pragma unroll 1
      for (int go = 0; go < (f32 ? 2 : 1); ++go) {
#pragma unroll 1
        for (int k = 0; k < (f32 ? 2 : 4); ++k) {   // 32 channels
          uint32_t o[32];
          if (some) {
            tmem_ld32(o_at + 64 * go + 32 * k, o);
            tmem_wait_ld();
          }
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = some ? __float_as_uint(__uint_as_float(o[j]) * inv) : 0u;
          auto put = [&](int c, uint4 w) { *reinterpret_cast<uint4*>(stage + lane * 256 + ((c ^ (lane & 15)) << 4)) = w; };
          if (f32) {
#pragma unroll
            for (int c = 0; c < 8; ++c) put(8 * k + c, make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]));
          } else {
            auto two = [&](int j) { return pack_in_dtype(__uint_as_float(o[j]), __uint_as_float(o[j + 1]), a.out_dtype); };
#pragma unroll
            for (int c = 0; c < 4; ++c) put(4 * k + c, make_uint4(two(8 * c), two(8 * c + 2), two(8 * c + 4), two(8 * c + 6)));
          }
        }
        __syncwarp();
        if (a.splits == 1 || some) {
#pragma unroll 4
          for (int k = 0; k < 16; ++k) {
            const int r = 2 * k + (lane >> 4), c = lane & 15, row = tid - lane + r;
            if (row < rows) {
              const uint4 w = *reinterpret_cast<const uint4*>(stage + r * 256 + ((c ^ (r & 15)) << 4));
              const long long at = a.splits > 1 ? row : out_row(row);
              reinterpret_cast<uint4*>(to + at * kD * (f32 ? 4 : 2) + 256 * go)[c] = w;
            }
          }
        }
        __syncwarp();
      }
      if (a.splits > 1 && tid < rows) {
        float* ml = part_ml(a, item) + 2 * tid;
        ml[0] = some ? mx : -INFINITY;
        ml[1] = some ? l : 0.0f;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // a wait of any role that ran out, the rows' last one too (their output is zeros then)
  if (tid == 0 && *flag) report(a.status, S4KV_ERR_DEVICE_TIMEOUT, S4KV_DEV_TIMEOUT, b);
  if (warp == kLoadWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmemCols));
}

// The splits of a row by the log-sum-exp rule: a CTA takes 32 rows of a tile and kv head, a
// warp four of them, a lane four channels.
__global__ void __launch_bounds__(256) prompt_join_kernel(PromptArgs a) {
  stream_wait();
  Place pl;
  if (find_tile<256, true>(a, blockIdx.x, pl) != kFound) return;
  const int h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cu0 = a.cu_q[pl.b], m = a.cu_q[pl.b + 1] - cu0;
  const long long item0 = (static_cast<long long>(blockIdx.x) * a.H + h) * a.splits;
  const int r0 = 32 * blockIdx.z + 4 * warp;
  const long long at0 = static_cast<long long>(pl.tile) * kQRows + r0, left = static_cast<long long>(m) * a.g - at0;
  if (left <= 0) return;
  const int n = left < 4 ? static_cast<int>(left) : 4;
  float w[4], inv[4];   // lane = part: its weight in row k; 1 / the row's sum
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float mi = -INFINITY, li = 0.0f;
    if (k < n && lane < a.splits) {
      const float2 ml = __ldcg(reinterpret_cast<const float2*>(part_ml(a, item0 + lane)) + r0 + k);
      mi = ml.x;
      li = ml.y;
    }
    const float M = warp_max(mi);
    // a part that saw nothing has l = 0 (and may have no rows at all); one with a NaN keeps it
    w[k] = li == 0.0f ? 0.0f : M == -INFINITY ? 1.0f : exp2_fast(mi - M);
    const float L = warp_sum(w[k] * li);
    if (li == 0.0f) w[k] = -1.0f;   // nothing to read
    inv[k] = L > 0.0f ? 1.0f / L : L == L ? 0.0f : L;
  }
  float4 o[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) o[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int s = 0; s < a.splits; ++s)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float ws = __shfl_sync(0xffffffffu, w[k], s);
      if (ws == -1.0f) continue;
      const float4 y = __ldcg(reinterpret_cast<const float4*>(part_rows(a, item0 + s) + (r0 + k) * kD) + lane);
      o[k] = make_float4(fmaf(ws, y.x, o[k].x), fmaf(ws, y.y, o[k].y), fmaf(ws, y.z, o[k].z), fmaf(ws, y.w, o[k].w));
    }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (k >= n) break;
    const float4 y = make_float4(o[k].x * inv[k], o[k].y * inv[k], o[k].z * inv[k], o[k].w * inv[k]);
    const long long at = at0 + k;
    const int i = static_cast<int>(at / a.g);
    const long long row = (static_cast<long long>(cu0) + i) * a.Hq + h * a.g + (at - static_cast<long long>(i) * a.g);
    if (a.out_dtype == S4KV_F32) {
      reinterpret_cast<float4*>(static_cast<float*>(a.out) + row * kD)[lane] = y;
    } else {
      reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row * kD)[lane] =
          make_uint2(pack_in_dtype(y.x, y.y, a.out_dtype), pack_in_dtype(y.z, y.w, a.out_dtype));
    }
  }
}

// Grants a kernel its shared memory on the current device, once per device.
template <bool CAP, bool SLOPE>
cudaError_t ready() {
  constexpr int kMaxDevices = 64;
  static std::mutex lock;
  static bool done[kMaxDevices] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> guard(lock);
  if (done[dev]) return cudaSuccess;
  const void* f = reinterpret_cast<const void*>(prompt_kernel<CAP, SLOPE>);
  cudaError_t e = prefer_max_shared(f);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return e;
  }
  done[dev] = true;
  return cudaSuccess;
}

template <bool CAP, bool SLOPE>
cudaError_t run(const PromptArgs& a, cudaStream_t st) {
  cudaError_t e = ready<CAP, SLOPE>();
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(a.q_tiles) * a.H, static_cast<unsigned>(a.splits));
  e = launch_behind(prompt_kernel<CAP, SLOPE>, grid, dim3(kThreads), kSmemBytes, st, a);
  if (e != cudaSuccess || a.splits == 1) return e;
  e = prefer_max_shared(reinterpret_cast<const void*>(prompt_join_kernel));
  if (e != cudaSuccess) return e;
  return launch_behind(prompt_join_kernel, dim3(static_cast<unsigned>(a.q_tiles), static_cast<unsigned>(a.H), kQRows / 32), dim3(256), 0, st, a);
}

}  // namespace

cudaError_t launch_prompt(const PromptArgs& a, cudaStream_t st) {
  if (a.form.cap > 0.0f) return a.form.slopes ? run<true, true>(a, st) : run<true, false>(a, st);
  return a.form.slopes ? run<false, true>(a, st) : run<false, false>(a, st);
}

}  // namespace s4kv
