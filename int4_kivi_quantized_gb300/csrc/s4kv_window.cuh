// Attention within a sliding window with sinks (s4kv_window_attention), on every
// page format, and all attention on INT8 block pages (a window wider than any
// sequence): the last nq tokens of each sequence as queries, nq >= 1. With SC, the
// same with a score form (s4kv_score_attention): the scores go through it behind their
// MMAs, and each query's visible tokens are a range of its own.
//
// The query at position p sees the tokens t <= p with t > p - W or t < S:
//   z_t = scale q . k_t,  P = softmax over the visible t,  out = sum_t P_t v_t.
// Decode attention reads each visible token's record once and does little with
// it, so the bound is the cache's bytes, and for short windows the latency of one
// pass through lengths, table, records and the combine.
//
// Units of work are blocks (32 tokens of KIVI pages, whose key metadata spans two
// pages; 16 tokens of the others). A (sequence, kv head, tile of query columns)
// segment has a list of blocks with a visible token: blocks that every query sees
// whole (sinks, then the window's inside) come first and run without masks, then
// the few that the window's start, the last sink, the queries' own positions or
// the residual cut. All segments' blocks form one line cut into equal slices, one
// per warp, as in decode attention; split segments leave partials that a second
// kernel, a programmatic dependent of the first, combines by the log-sum-exp rule.
// Consecutive slices go to different SMs, so a small call spreads over the GPU.
//
//  * 8-bit pages: a warp streams records through a ring of stages (bulk copies,
//    bounded waits). Scores take the query columns as MMA rows, so what a lane
//    ends with is the operand of P V. An INT8 code enters an MMA as the f16
//    subnormal (c + 128) 2^-24, one byte permute for two codes and no arithmetic;
//    128 times the query's sum comes off the scores, and the P V accumulators
//    start at -128 2^-24 times the sum of the rounded P (one MMA against a
//    constant tile), so what a block adds is exact codes times its own fp32 scale.
//    In a cut block a token that no query sees may have set the scale (the type's
//    largest value, say), and a rest of those subtractions times it would be felt:
//    there the codes enter as the signed numbers that they are.
//  * KIVI pages: the key scales are folded into the query and the minima into a
//    bias per column, the value scales into P and the minima into a bias per column
//    and channel group, 8 columns a warp; cut blocks and the residual go through a
//    masked form of the decode kernel's tail.
//
// Measured (GB300, a captured graph's time a call; bytes: the visible records, rings,
// queries and outputs at the rate of a plain copy, 6783 GB/s): INT8 pages, one sequence
// of 256 tokens, one kv head 6.4 us (latency); 8 kv heads of 4 queries, 32 sequences of
// 1024 to 8192 tokens 54.5 (bytes 44.8); 16 of 777 to 8191 with four query positions 39.5
// (21.9: 16 columns leave three warps a scheduler, and each waits on its own chain of
// score, exponential and value MMAs); 32 of 32768, 4 kv heads of 7 queries, 167 (158.7).
// 64 sequences behind a window of 4096, 8 kv heads: 4-bit pages 82.5 (61.3), 2-bit 81
// (41.8), FP8 92.5 (79.4), INT8 89.5 (79.7). On 4- and 2-bit pages that is the arithmetic of
// the codes, and the cut blocks of each segment, which go one by one and wait for their own
// loads: the sinks', the window's first, and those that the residual reaches (five of them
// at R = 128), about an eighth of the work line. Outputs in 32 bits take the same times.
//
// With a score form, the same launches cost 3 to 9% more (times without, with a window as a form, and with
// a cap and slopes): INT8, 16 sequences of 4096 tokens with four queries each, 8 kv heads 31.7, 34.4, 37.1 us; 64 of
// 2000 with one query 4-bit 49.5, 51.3, 53.6, FP8 52.6, 55.4, 57.5, INT8 47.3, 48.7, 49.6; one sequence of 256
// 6.4, 6.8, 6.8. A capped 4-bit decode of 32 contexts of 32768 (28 heads) 155 us against 142: the cubic
// near zero is three packed multiply-adds and two products for two scores where the exponential
// form is two special instructions a score, 166 us. Slopes are one multiply-add a score.
//
// A masked token's key and value never meet arithmetic that could carry an
// infinity or a NaN of theirs into the result: scores are selected, probabilities
// scaled only where they are positive, 16-bit and FP8 value rows that no column
// sees read as zeros, and where columns of one tile see different tokens and such
// a row is not finite, the block is done query by query.

#pragma once

#include "s4kv_kernels.cuh"
#include "s4kv_score.cuh"

#include <mutex>
#include <type_traits>

namespace s4kv {
namespace {

constexpr int kI8 = S4KV_BITS_INT8;
// Warps of a CTA (one CTA per SM), and the records that a warp of 8-bit pages has in
// flight or at hand. More warps would hide more of a page's latency, but 16 columns
// then spill (16 sequences of 777 to 8191 tokens, 8 kv heads: 16 warps of 128 registers
// 54 us, 12 warps 44); more records do not help INT8 pages, whose loads outrun the arithmetic: three for
// each of 12 warps, 22 MB in flight over the GPU, read 16 sequences of 32000 tokens,
// 8 kv heads, in 175 us, two in 166 us, and 8 to 16 warps with two to four lie between.
constexpr int kWarps = 12;
template <int FMT> constexpr int kStagesOf = FMT == kI8 ? 2 : 3;
template <int FMT> constexpr bool kByte = FMT == 8 || FMT == kI8;
template <int FMT> constexpr int kBlock = kByte<FMT> ? kP : kG;             // tokens of a block
// 8-bit pages: the stages, or a warp's 16 columns of output when a segment is combined
template <int FMT, int NC> constexpr int kRegionOf = kByte<FMT> ? (kStagesOf<FMT> * Rec<kI8>::kBytes > 16 * kD * 4 ? (kStagesOf<FMT> * Rec<kI8>::kBytes + 127) / 128 * 128 : 16 * kD * 4) : kRegion;
template <int FMT> constexpr int kLeastUnits = kByte<FMT> ? 4 : 3;           // least work per warp
// Behind the blocks of a segment the line has kSegCost positions without work: a warp
// that goes on to another segment writes a partial and starts again at the lengths and
// the table, which takes it some blocks' time. 8-bit pages: 0 / 4 / 6 / 12 blocks: 32
// sequences of 1024 to 8192 tokens 57.6 / 55.7 / 55.9 / 56.2 us, 16 of 777 to 8191 with
// 16 columns 44.4 / 40.7 / 39.1 / 38.9. KIVI pages, where the cut blocks' cost says it
// already: 0 / 1 / 3: 64 sequences behind a window of 4096 83.8 / 84.1 / 85.4.
template <int FMT> constexpr int kSegCost = kByte<FMT> ? 6 : 0;
// With a score form the unfinished block of INT8 pages counts as so many records: its 16-bit rows
// come by plain loads, 7500 cycles where a record takes 2500.
constexpr int kRingUnits = 4;

template <int FMT, int NC, bool SC>
struct WSmem {
  alignas(128) uint8_t region[kWarps][kRegionOf<FMT, NC>];
  alignas(16) float ptile[kByte<FMT> ? 1 : kWarps][32 * kPRow];
  alignas(16) uint4 q[NC == 16 ? kWarps : 1][NC == 16 ? 8 : 1][32];   // 16 columns: the queries as A operands, by slice and lane
  float zscale[NC == 16 ? kWarps : 1][NC == 16 ? 16 : 1];   // and their score scales, by column
  // a segment's slopes by column, times log2 e, and its queries' spans (KIVI pages: in the P
  // tile's rows, which leave four floats each, see kSpanAt)
  float slope2[SC && kByte<FMT> ? kWarps : 1][SC && kByte<FMT> ? 16 : 1];
  Span spans[SC && kByte<FMT> ? kWarps : 1][SC && kByte<FMT> ? 16 : 1];
  alignas(8) uint64_t bar[kWarps][4];
};
// Behind it: the cost prefix of the line (int64 [B + 1]), or what a one-segment
// launch combines: each warp's maxima and sums, then the CTA's own state.
struct OneSmem {
  float wm[kWarps][16], wl[kWarps][16];
  alignas(16) float part[16][kD];
  float pm[16], pl[16];
};
template <int FMT, int NC, bool SC>
__host__ __device__ constexpr size_t prefix_at() { return (sizeof(WSmem<FMT, NC, SC>) + 15) / 16 * 16; }
static_assert(prefix_at<4, 8, true>() + 4097 * sizeof(long long) <= 227 * 1024 &&
                  prefix_at<4, 8, true>() + sizeof(OneSmem) <= 227 * 1024,
              "the largest batch fits the shared memory of a CTA");

// The kernel's arguments: with SC, those of a score form too.
template <bool SC> using Args = std::conditional_t<SC, ScoredArgs, WindowArgs>;

// What a masked block needs to know: its first token, the tile's first and last query
// position. SC: every query's span (spans[position - base]), and the hull of the tile's.
struct Cut {
  int tok0, window, sinks, first, last;
  const float* spans;   // `step` floats apart
  int step, base, lo, hi;
  __device__ __forceinline__ Span span(int pos) const { return *reinterpret_cast<const Span*>(spans + (pos - base) * step); }
};
// KIVI pages: where a query's span and a column's slope sit in row i of the warp's P tile.
constexpr int kSpanAt = 8, kSlopeAt = 10;
static_assert(kPRow >= 11 && kPRow % 2 == 0, "a span and a slope fit behind a row of P");
template <bool SC>
__device__ __forceinline__ bool visible(int t, int pos, const Cut& cut) {
  if constexpr (SC) return sees(cut.span(pos), t, cut.sinks);
  else return t <= pos && (t > pos - cut.window || t < cut.sinks);
}
// Whether a query at one of the positions [lo, hi] (one position, or all of the tile's) may see t.
template <bool SC>
__device__ __forceinline__ bool visible_to(int t, int lo, int hi, const Cut& cut) {
  if constexpr (SC) {
    if (lo == hi) return visible<SC>(t, lo, cut);
    return t <= cut.hi && (t >= cut.lo || t < cut.sinks);
  } else {
    return t <= hi && (t > lo - cut.window || t < cut.sinks);
  }
}
// Whether the query at `pos` sees any of the n tokens from cut.tok0 on.
template <bool SC>
__device__ __forceinline__ bool visible_block(int n, int pos, const Cut& cut) {
  if constexpr (SC) {
    const Span s = cut.span(pos);
    return (max(cut.tok0, s.lo) <= min(cut.tok0 + n - 1, s.hi)) || (cut.tok0 < cut.sinks && cut.tok0 <= s.hi);
  } else {
    return cut.tok0 <= pos && (cut.tok0 + n - 1 > pos - cut.window || cut.tok0 < cut.sinks);
  }
}

// Scores z in log2 units through the form: capped, less slope2 |rel - on(i)|, rel the query's position
// less a token, on(i) how far behind that one z[i]'s token is. Called by the whole warp.
__device__ __forceinline__ float lane_token(int x) { return (x & 1) + 8.0f * (x >> 1); }   // of a lane's four tokens
template <int N, class ON>
__device__ __forceinline__ void through_form(float (&z)[N], const ScoredArgs& a, float slope2, int rel, ON on) {
  static_assert(N % 2 == 0, "scores in pairs");
  if (a.cap2 > 0.0f) {
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) top = fmaxf(top, fabsf(z[i]));
    if (__all_sync(0xffffffffu, top <= kNearCap * a.cap2)) {
      const float2 by = make_float2(a.icap2, a.icap2);
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const float2 x = make_float2(z[i], z[i + 1]), u = __fmul2_rn(x, by), w = __fmul2_rn(u, u);
        float2 p = make_float2(near_coef(kNearCoefs - 1), near_coef(kNearCoefs - 1));
#pragma unroll
        for (int k = kNearCoefs - 2; k >= 0; --k) p = __ffma2_rn(p, w, make_float2(near_coef(k), near_coef(k)));
        p = __fmul2_rn(x, p);
        z[i] = p.x;
        z[i + 1] = p.y;
      }
    } else {
      const float by = a.icap2 * 2.8853900817779268f;   // 2 log2(e)
#pragma unroll
      for (int i = 0; i < N; ++i) z[i] = far_cap(z[i], by, a.cap2);
    }
  }
  if (a.score.slopes) {
    const float from = static_cast<float>(rel);
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = fmaf(-slope2, fabsf(from - on(i)), z[i]);
  }
}

// Visible blocks of a sequence of T tokens: whole ones [0, A0) and [F0, F1), cut
// ones [A0, A1), [W0, F0) and [F1, E). One plan serves every tile of the sequence.
template <int FMT>
struct Plan {
  int A0, A1, W0, F0, F1, E, nf, nx;
  long long work;   // cost of the blocks; kSegCost positions without any follow
  __device__ __forceinline__ long long cost() const { return work + kSegCost<FMT>; }
  __device__ __forceinline__ int block_of(int u) const {   // unit u: whole blocks first
    if (u < A0) return u;
    if (u < nf) return F0 + u - A0;
    u -= nf;
    if (u < A1 - A0) return A0 + u;
    u -= A1 - A0;
    if (u < F0 - W0) return W0 + u;
    return F1 + u - (F0 - W0);
  }
};

// Of the spans of a tile's queries: the earliest and the latest start, the earliest end (the latest is T - 1).
struct Reach {
  int w_first, w_last, end;
  __device__ __forceinline__ void add(const Span& s, int T) {
    w_first = min(w_first, s.lo);
    w_last = max(w_last, min(s.lo, T));
    end = min(end, s.hi);
  }
};
template <int FMT, bool SC>
__device__ __forceinline__ Plan<FMT> plan_by(int T, const Args<SC>& a, const Reach& r) {
  constexpr int BT = kBlock<FMT>;
  Plan<FMT> p;
  if (T < a.nq || T <= 0 || T > a.max_seq_len) {   // nothing to attend to (T = 0), or a bad length
    p.A0 = p.A1 = p.W0 = p.F0 = p.F1 = p.E = p.nf = p.nx = 0;
    p.work = 1;
    return p;
  }
  // blocks that are quantized whole
  const int main = FMT == kI8 ? T / BT : FMT == 8 ? T / BT : (min(T & ~(kG - 1), max(0, T - a.R)) / kG);
  p.E = (T - 1) / BT + 1;
  p.W0 = r.w_first / BT;
  p.A1 = min((a.sinks + BT - 1) / BT, p.W0);
  p.A0 = min(min(a.sinks / BT, p.A1), main);
  if constexpr (SC) p.A0 = min(p.A0, (r.end + 1) / BT);
  p.F0 = (r.w_last + BT - 1) / BT;
  p.F1 = min(main, (r.end + 1) / BT);
  if (p.F0 >= p.F1) p.F0 = p.F1 = p.W0;
  p.nf = p.A0 + p.F1 - p.F0;
  p.nx = (p.A1 - p.A0) + (p.F0 - p.W0) + (p.E - p.F1);
  p.work = p.nf + static_cast<long long>(kByte<FMT> ? 1 : a.tail_cost) * p.nx;
  if (SC && FMT == kI8 && T % BT != 0) p.work += kRingUnits - 1;
  return p;
}

// The plan of sequence b, by one thread.
template <int FMT, bool SC>
__device__ __forceinline__ Plan<FMT> plan_of(int T, const Args<SC>& a, int b) {
  const int first = T - a.nq;                               // position of the first query
  if constexpr (SC) {
    Reach r{T - 1, 0, T - 1};
#pragma unroll 4
    for (int i = 0; i < a.nq; ++i) r.add(span_of(a.score, first + i, T, static_cast<long long>(b) * a.nq + i, b), T);
    return plan_by<FMT, SC>(T, a, r);
  } else {
    return plan_by<FMT, SC>(T, a, Reach{max(0, first - a.window + 1), max(0, T - a.window), first});
  }
}
// By a whole warp, a query a lane; `mine`: the span of the lane's.
template <int FMT, bool SC>
__device__ __forceinline__ Plan<FMT> plan_of_warp(int T, const Args<SC>& a, int b, Span& mine) {
  mine = Span{0x7fffffff, -1};
  if constexpr (SC) {
    const int lane = threadIdx.x & 31;
    Reach r{T - 1, 0, T - 1};
    if (lane < a.nq) {
      mine = span_of(a.score, T - a.nq + lane, T, static_cast<long long>(b) * a.nq + lane, b);
      r.add(mine, T);
    }
    r.w_first = __reduce_min_sync(0xffffffffu, r.w_first);
    r.w_last = __reduce_max_sync(0xffffffffu, r.w_last);
    r.end = __reduce_min_sync(0xffffffffu, r.end);
    return plan_by<FMT, SC>(T, a, r);
  } else {
    return plan_of<FMT, SC>(T, a, b);
  }
}

__device__ __forceinline__ void mma16816_c(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1,
                                           const float (&c)[4]) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

// ---- 8-bit pages -------------------------------------------------------------------------

// State of a warp's NC columns: column 8 ct + gi is row r = ct of m and l (this
// lane's part of the sum); o[mt][ct] holds columns 8 ct + 2ti, + 2ti + 1 of the
// channels that rows gi and gi + 8 of tile mt stand for.
template <int NC>
struct ByteState {
  static constexpr int CT = NC / 8;
  float o[8][CT][4];
  float m[CT], l[CT];
};

template <int NC>
__device__ __forceinline__ void byte_init(ByteState<NC>& s) {
#pragma unroll
  for (int c = 0; c < NC / 8; ++c) {
    s.m[c] = -INFINITY;
    s.l[c] = 0.0f;
#pragma unroll
    for (int mt = 0; mt < 8; ++mt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s.o[mt][c][e] = 0.0f;
  }
}

// Online softmax over 16 tokens: z[ct][x], x = tokens 2ti, 2ti+1, 2ti+8, 2ti+9 of
// the block (-inf: masked), becomes p; accumulators are rescaled when a maximum
// rises by more than kLazy. kMask: a column may have seen nothing so far.
template <int NC, bool kMask>
__device__ __forceinline__ void byte_softmax(ByteState<NC>& s, float (&z)[NC / 8][4]) {
  constexpr int CT = NC / 8;
  const int ti = threadIdx.x & 3;
  float mx[CT];
  bool up = false;
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    mx[c] = fmaxf(fmaxf(z[c][0], z[c][1]), fmaxf(z[c][2], z[c][3]));
    up = up || mx[c] > s.m[c] + kLazy;
  }
  if (__any_sync(0xffffffffu, up)) {   // rare: only now the lanes of a column agree on its maximum
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      mx[c] = fmaxf(mx[c], __shfl_xor_sync(0xffffffffu, mx[c], 1));
      mx[c] = fmaxf(mx[c], __shfl_xor_sync(0xffffffffu, mx[c], 2));
      const float mn = fmaxf(s.m[c], mx[c]);
      const float al = mn == -INFINITY ? 1.0f : ex2(s.m[c] - mn);
      s.m[c] = mn;
      s.l[c] *= al;
      // output columns 8c + 2ti and + 1 keep their state in lanes 8ti and 8ti + 4
      const float a0 = __shfl_sync(0xffffffffu, al, 8 * ti), a1 = __shfl_sync(0xffffffffu, al, 8 * ti + 4);
#pragma unroll
      for (int mt = 0; mt < 8; ++mt) {
        s.o[mt][c][0] *= a0;
        s.o[mt][c][1] *= a1;
        s.o[mt][c][2] *= a0;
        s.o[mt][c][3] *= a1;
      }
    }
  }
#pragma unroll
  for (int c = 0; c < CT; ++c) {
#pragma unroll
    for (int x = 0; x < 4; ++x) z[c][x] = kMask && z[c][x] == -INFINITY ? 0.0f : ex2(z[c][x] - s.m[c]);
    s.l[c] += (z[c][0] + z[c][1]) + (z[c][2] + z[c][3]);
  }
}

// Adds a product to the accumulator columns of one position only (columns 2ti and
// 2ti + 1 have positions opos): where a value row is not finite, the other
// columns' zeros would meet it.
template <class F>
__device__ __forceinline__ void add_only(float (&o)[4], const int (&opos)[2], int only, F product) {
  float t[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  product(t);
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = opos[e & 1] == only ? o[e] + t[e] : o[e];
}

// What INT8 accumulators lack of the true output, until the records are done.
constexpr float kI8Rest = 262144.0f;

// INT8 codes as exact f16 numbers: byte | 0x6400 is 1024 + byte, less 1152.
__device__ __forceinline__ uint32_t less1152(uint32_t w) {
  const uint32_t k = 0x64806480u;
  const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&w), *reinterpret_cast<const __half2*>(&k));
  return *reinterpret_cast<const uint32_t*>(&d);
}
__device__ __forceinline__ uint32_t codes01(uint32_t w) { return less1152(__byte_perm(w, 0x64646464u, 0x4140)); }
__device__ __forceinline__ uint32_t codes23(uint32_t w) { return less1152(__byte_perm(w, 0x64646464u, 0x4342)); }

// One staged record of 16 tokens. Keys: lane (gi, ti) reads its words as the B
// operand of tokens gi and gi + 8; q as A. qa: f16 queries, rows gi (and gi + 8), each
// column at a power of two of its own (query_power); zscale[ct] = sm_scale log2(e) over
// that power, times the key scale (FP8) or the 2^24 of the codes' subnormals (INT8), and
// zoff[ct] = -128 scale sum_c q_c (INT8).
// Sixteen columns leave no registers for the queries and their scales: qs and zs hold
// them (32 sequences of 1024 to 8192 tokens, 16 query tokens: 197.5 us, scales in registers
// 199.6). kMask: tokens are masked by `cut` and the columns' positions.
template <int FMT, int NC, bool kMask, bool SC>
__device__ __forceinline__ void byte_block(const Args<SC>& args, const char* rec, ByteState<NC>& s, const uint32_t (&qa)[8][2],
                                           const uint4 (*qs)[32], const float (&zoff)[NC / 8], float zscale0, const float* zs,
                                           const float* slope2, const Cut& cut, const int (&pos)[NC / 8],
                                           const int (&opos)[NC / 8][2]) {
  constexpr int CT = NC / 8;
  const int lane = threadIdx.x & 31, ti = lane & 3;
  float z[CT][4];
  float vscale = 1.0f;
  float zscale[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) zscale[c] = NC == 16 ? zs[8 * c + (lane >> 2)] : zscale0;
  {
    // two chains of four MMAs for each eight tokens instead of one of eight
    float s0[4] = {0.0f, 0.0f, 0.0f, 0.0f}, s1[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    float u0[4] = {0.0f, 0.0f, 0.0f, 0.0f}, u1[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int kp = 0; kp < 4; ++kp) {
      const uint4 w = *reinterpret_cast<const uint4*>(rec + kp * 512 + lane * 16);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t w0 = u ? w.z : w.x, w1 = u ? w.w : w.y;
        const int kk = 2 * kp + u;
        uint32_t a[4] = {qa[kk][0], 0u, qa[kk][1], 0u};
        if constexpr (NC == 16) {
          const uint4 x = qs[kk][lane];
          a[0] = x.x;
          a[1] = x.y;
          a[2] = x.z;
          a[3] = x.w;
        }
        if constexpr (FMT == kI8 && kMask) {
          mma16816(u ? u0 : s0, a, codes01(w0), codes01(w1));
          mma16816(u ? u1 : s1, a, codes23(w0), codes23(w1));
        } else if constexpr (FMT == kI8) {
          mma16816(u ? u0 : s0, a, __byte_perm(w0, 0u, 0x4140), __byte_perm(w1, 0u, 0x4140));
          mma16816(u ? u1 : s1, a, __byte_perm(w0, 0u, 0x4342), __byte_perm(w1, 0u, 0x4342));
        } else {
          mma16816(u ? u0 : s0, a, fp8x2_to_f16x2(w0 & 0xffffu), fp8x2_to_f16x2(w1 & 0xffffu));
          mma16816(u ? u1 : s1, a, fp8x2_to_f16x2(w0 >> 16), fp8x2_to_f16x2(w1 >> 16));
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s0[i] += u0[i];
      s1[i] += u1[i];
    }
    if constexpr (FMT == kI8) {
      const float2 sc = *reinterpret_cast<const float2*>(rec + Rec<kI8>::kKs);
      vscale = sc.y;
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        const float c1 = sc.x * (kMask ? zscale[c] * (1.0f / 16777216.0f) : zscale[c]);
        const float c2 = kMask ? 0.0f : sc.x * zoff[c];
        z[c][0] = fmaf(s0[2 * c], c1, c2);
        z[c][1] = fmaf(s0[2 * c + 1], c1, c2);
        z[c][2] = fmaf(s1[2 * c], c1, c2);
        z[c][3] = fmaf(s1[2 * c + 1], c1, c2);
      }
    } else {
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        z[c][0] = s0[2 * c] * zscale[c];
        z[c][1] = s0[2 * c + 1] * zscale[c];
        z[c][2] = s1[2 * c] * zscale[c];
        z[c][3] = s1[2 * c + 1] * zscale[c];
      }
    }
  }
  bool sees[CT][4];
  if (kMask) {
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        sees[c][x] = visible<SC>(cut.tok0 + 2 * ti + (x & 1) + 8 * (x >> 1), pos[c], cut);
        // (what an FP8 page holds behind the last token has no say in how the others are capped)
        if (SC && !sees[c][x]) z[c][x] = 0.0f;
      }
  }
  if constexpr (SC) {
#pragma unroll
    for (int c = 0; c < CT; ++c)
      through_form(z[c], args, slope2[8 * c + (lane >> 2)], pos[c] - cut.tok0 - 2 * ti, lane_token);
  }
  if (kMask) {
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int x = 0; x < 4; ++x) z[c][x] = sees[c][x] ? z[c][x] : -INFINITY;
  }
  byte_softmax<NC, kMask>(s, z);
  uint32_t b[CT][2];
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    b[c][0] = pack_f16x2(z[c][0], z[c][1]);
    b[c][1] = pack_f16x2(z[c][2], z[c][3]);
  }
  if constexpr (FMT == kI8) {
    float bias[CT][4], f[CT][2];
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      // -2^-17 = -128 2^-24 in every element (f16 subnormal 0x8080)
      const uint32_t k[4] = {0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u};
      const float zero[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      if constexpr (kMask) {
#pragma unroll
        for (int e = 0; e < 4; ++e) bias[c][e] = 0.0f;
      } else {
        mma16816_c(bias[c], k, b[c][0], b[c][1], zero);
      }
      // 2^24 of the codes' subnormals: 2^6 here, so that no scale overflows, and kI8Rest at the end
      const float vs = vscale * (kMask ? 1.0f / kI8Rest : 16777216.0f / kI8Rest);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        bool any = true;
        if (kMask) any = visible_block<SC>(kP, opos[c][e], cut);
        f[c][e] = any ? vs : 0.0f;
      }
    }
#pragma unroll
    for (int kp = 0; kp < 4; ++kp) {
      const uint4 w = *reinterpret_cast<const uint4*>(rec + 2048 + kp * 512 + lane * 16);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t w0 = u ? w.z : w.x, w1 = u ? w.w : w.y;
        uint32_t a[4];
        if constexpr (kMask) {
          a[0] = codes01(w0);
          a[1] = codes23(w0);
          a[2] = codes01(w1);
          a[3] = codes23(w1);
        } else {
          a[0] = __byte_perm(w0, 0u, 0x4140);
          a[1] = __byte_perm(w0, 0u, 0x4342);
          a[2] = __byte_perm(w1, 0u, 0x4140);
          a[3] = __byte_perm(w1, 0u, 0x4342);
        }
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          float t[4];
          mma16816_c(t, a, b[c][0], b[c][1], bias[c]);
          float(&o)[4] = s.o[2 * kp + u][c];
          o[0] = fmaf(t[0], f[c][0], o[0]);
          o[1] = fmaf(t[1], f[c][1], o[1]);
          o[2] = fmaf(t[2], f[c][0], o[2]);
          o[3] = fmaf(t[3], f[c][1], o[3]);
        }
      }
    }
  } else {
    uint4 vw[4];
#pragma unroll
    for (int kp = 0; kp < 4; ++kp) vw[kp] = *reinterpret_cast<const uint4*>(rec + 2048 + kp * 512 + lane * 16);
    // only: the position whose columns take the product, -1 for all
    auto pv = [&](uint32_t m01, uint32_t m23, int only) {
#pragma unroll
      for (int mt = 0; mt < 8; ++mt) {
        const uint32_t w0 = (mt & 1) ? vw[mt >> 1].z : vw[mt >> 1].x, w1 = (mt & 1) ? vw[mt >> 1].w : vw[mt >> 1].y;
        uint32_t a[4] = {fp8x2_to_f16x2(w0 & 0xffffu), fp8x2_to_f16x2(w0 >> 16), fp8x2_to_f16x2(w1 & 0xffffu),
                         fp8x2_to_f16x2(w1 >> 16)};
        if (kMask) {
          a[0] &= m01;
          a[1] &= m01;
          a[2] &= m23;
          a[3] &= m23;
        }
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          if (!kMask || only < 0) mma16816(s.o[mt][c], a, b[c][0], b[c][1]);
          else add_only(s.o[mt][c], opos[c], only, [&](float (&t)[4]) { mma16816(t, a, b[c][0], b[c][1]); });
        }
      }
    };
    if constexpr (!kMask) {
      pv(0xffffffffu, 0xffffffffu, -1);
    } else {
      // halves of the tokens 2ti, 2ti+1 | 2ti+8, 2ti+9 that a query at one of the
      // positions [lo, hi] sees
      auto halves = [&](int lo, int hi, uint32_t& m01, uint32_t& m23) {
        uint32_t m[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int t = cut.tok0 + 2 * ti + (x & 1) + 8 * (x >> 1);
          m[x] = visible_to<SC>(t, lo, hi, cut) ? 0xffffu : 0u;
        }
        m01 = m[0] | (m[1] << 16);
        m23 = m[2] | (m[3] << 16);
      };
      bool nan = false;   // an e4m3 NaN byte
      if (cut.first != cut.last) {
#pragma unroll
        for (int kp = 0; kp < 4; ++kp) {
          const uint32_t w[4] = {vw[kp].x, vw[kp].y, vw[kp].z, vw[kp].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) nan = nan || (((w[i] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u);
        }
      }
      if (!__any_sync(0xffffffffu, nan)) {
        uint32_t m01, m23;
        halves(cut.first, cut.last, m01, m23);
        pv(m01, m23, -1);
      } else {
        for (int q = cut.first; q <= cut.last; ++q) {
          uint32_t m01, m23;
          halves(q, q, m01, m23);
          pv(m01, m23, q);
        }
      }
    }
  }
}

template <int DT>
__device__ __forceinline__ void mma_in(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (DT == S4KV_BF16) mma16816_bf16(d, a, b0, b1);
  else mma16816(d, a, b0, b1);
}
template <int DT>
__device__ __forceinline__ uint32_t pack_in(float lo, float hi) {
  if constexpr (DT == S4KV_BF16) return pack_bf16x2(lo, hi);
  else return pack_f16x2(lo, hi);
}
template <int DT>
__device__ __forceinline__ float2 unpack_in(uint32_t w) {
  if constexpr (DT == S4KV_BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  else return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
// Whether a packed 16-bit pair holds an infinity or a NaN.
template <int DT>
__device__ __forceinline__ bool wild(uint32_t w) {
  constexpr uint32_t e = DT == S4KV_BF16 ? 0x7f80u : 0x7c00u;
  return (w & e) == e || (w & (e << 16)) == (e << 16);
}

// The unfinished block of INT8 pages: n tokens from tok0 on, 16-bit rows of the
// rings, read from global memory straight into operands (exact products with the
// query in its own type, P split into two 16-bit terms).
template <int DT, int NC, bool SC>
__device__ __forceinline__ void ring_block(const Args<SC>& args, const uint16_t* kring, const uint16_t* vring, int n, ByteState<NC>& s,
                                           const uint16_t* (&qrow)[NC / 8], float scale, const float* slope2, const Cut& cut,
                                           const int (&pos)[NC / 8], const int (&opos)[NC / 8][2]) {
  constexpr int CT = NC / 8;
  const int lane = threadIdx.x & 31, gi = lane >> 2, ti = lane & 3;
  const uint4 none = make_uint4(0u, 0u, 0u, 0u);
  uint4 v[4][2];
  bool part = false;   // a row some columns see and others do not, that is not finite
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const int t = 2 * ti + (x & 1) + 8 * (x >> 1), at = cut.tok0 + t;
    const bool any = t < n && visible_to<SC>(at, cut.first, cut.last, cut);
    const uint4* row = reinterpret_cast<const uint4*>(vring + t * kD);
    v[x][0] = any ? row[gi] : none;
    v[x][1] = any ? row[gi + 8] : none;
  }
  float z[CT][4];
  {
    float s0[4] = {0.0f, 0.0f, 0.0f, 0.0f}, s1[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < 4; ++j) {   // channels 32 ti + 8 j .. + 7
      const uint4 k0 = gi < n ? reinterpret_cast<const uint4*>(kring + gi * kD)[4 * ti + j] : none;
      const uint4 k1 = gi + 8 < n ? reinterpret_cast<const uint4*>(kring + (gi + 8) * kD)[4 * ti + j] : none;
      uint4 q[2] = {none, none};
#pragma unroll
      for (int c = 0; c < CT; ++c)
        if (qrow[c]) q[c] = reinterpret_cast<const uint4*>(qrow[c])[4 * ti + j];
      const uint32_t a0[4] = {q[0].x, q[1].x, q[0].y, q[1].y}, a1[4] = {q[0].z, q[1].z, q[0].w, q[1].w};
      mma_in<DT>(s0, a0, k0.x, k0.y);
      mma_in<DT>(s0, a1, k0.z, k0.w);
      mma_in<DT>(s1, a0, k1.x, k1.y);
      mma_in<DT>(s1, a1, k1.z, k1.w);
    }
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      z[c][0] = s0[2 * c] * scale;
      z[c][1] = s0[2 * c + 1] * scale;
      z[c][2] = s1[2 * c] * scale;
      z[c][3] = s1[2 * c + 1] * scale;
      bool sees[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        sees[x] = visible<SC>(cut.tok0 + 2 * ti + (x & 1) + 8 * (x >> 1), pos[c], cut);
        if (SC && !sees[x]) z[c][x] = 0.0f;   // (no say in how the others are capped)
      }
      if constexpr (SC)
        through_form(z[c], args, slope2[8 * c + gi], pos[c] - cut.tok0 - 2 * ti, lane_token);
#pragma unroll
      for (int x = 0; x < 4; ++x) z[c][x] = sees[x] ? z[c][x] : -INFINITY;
    }
  }
  byte_softmax<NC, true>(s, z);
  uint32_t hi[CT][2], lo[CT][2];
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      hi[c][e] = pack_in<DT>(z[c][2 * e], z[c][2 * e + 1]);
      const float2 r = unpack_in<DT>(hi[c][e]);
      lo[c][e] = pack_in<DT>(z[c][2 * e] - r.x, z[c][2 * e + 1] - r.y);
    }
  if (cut.first != cut.last) {
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        part = part || wild<DT>(v[x][e].x) || wild<DT>(v[x][e].y) || wild<DT>(v[x][e].z) || wild<DT>(v[x][e].w);
  }
  auto pv = [&](const bool (&keep)[4], int only) {   // only: as in byte_block
#pragma unroll
    for (int mt = 0; mt < 8; ++mt) {
      const uint32_t sel = (mt & 1) ? 0x7632u : 0x5410u;
      uint32_t w[4][2];
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint4& y = v[x][e];
          const uint32_t u = (mt >> 1) == 0 ? y.x : (mt >> 1) == 1 ? y.y : (mt >> 1) == 2 ? y.z : y.w;
          w[x][e] = keep[x] ? u : 0u;
        }
      const uint32_t a[4] = {__byte_perm(w[0][0], w[1][0], sel), __byte_perm(w[0][1], w[1][1], sel),
                             __byte_perm(w[2][0], w[3][0], sel), __byte_perm(w[2][1], w[3][1], sel)};
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        auto product = [&](float (&t)[4]) {
          mma_in<DT>(t, a, hi[c][0], hi[c][1]);
          mma_in<DT>(t, a, lo[c][0], lo[c][1]);
        };
        if (only < 0) product(s.o[mt][c]);
        else add_only(s.o[mt][c], opos[c], only, product);
      }
    }
  };
  if (!__any_sync(0xffffffffu, part)) {
    const bool all[4] = {true, true, true, true};
    pv(all, -1);
  } else {
    for (int q = cut.first; q <= cut.last; ++q) {
      bool keep[4];
#pragma unroll
      for (int x = 0; x < 4; ++x)
        keep[x] = visible<SC>(cut.tok0 + 2 * ti + (x & 1) + 8 * (x >> 1), q, cut);
      pv(keep, q);
    }
  }
}

// ---- KIVI pages: a whole block (32 tokens, both page records in `stage`) -----------------
// As on 8-bit pages the query columns are the MMA's rows: a lane's code words are the
// B operand of tokens gi and gi + 8 as they stand (f16 subnormals), and A holds
// q' = q * scale of column gi in rows 0..7 and what its rounding to f16 left in rows
// 8..15, so one MMA carries both terms for eight columns and a lane adds its own two
// rows. The scores are then the operand of P V already: no pass through shared
// memory. (m, l): state of column gi; s.o and s.bias as the decode kernel has them
// (o at the powers of two that mma_unscale removes).
// SC: rel, the column's position less the block's first token, and its slope.
template <int BITS, bool SC>
__device__ __forceinline__ void kivi_block(const Args<SC>& args, const char* stage, MmaState& s, float& m, float& l,
                                           const float (&q)[32], float scale, int rel, float slope2) {
  using F = Rec<BITS>;
  constexpr int RS = kRecStrideB<BITS>;
  const int lane = threadIdx.x & 31, ti = lane & 3;
  uint32_t w[2][8];
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const uint4 x = *reinterpret_cast<const uint4*>(stage + p * RS + F::kKc + lane * 16);
    w[p][0] = x.x; w[p][1] = x.y; w[p][2] = x.z; w[p][3] = x.w;
    if constexpr (BITS == 4) {
      const uint4 y = *reinterpret_cast<const uint4*>(stage + p * RS + F::kKc + 512 + lane * 16);
      w[p][4] = y.x; w[p][5] = y.y; w[p][6] = y.z; w[p][7] = y.w;
    }
  }
  float c[4][4];   // page p, tokens 0..7 | 8..15: c[2p + half]
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) c[i][e] = 0.0f;
  float2 beta2 = make_float2(0.0f, 0.0f);
  const char* mrec = stage + (ti >> 1) * RS + F::kKm + (ti & 1) * 16;
#pragma unroll
  for (int kk = 0; kk < 8; ++kk) {
    const float4 s4 = *reinterpret_cast<const float4*>(mrec + kk * 32), m4 = *reinterpret_cast<const float4*>(mrec + kk * 32 + 256);
    const float2 q01 = make_float2(q[4 * kk], q[4 * kk + 1]), q23 = make_float2(q[4 * kk + 2], q[4 * kk + 3]);
    beta2 = __ffma2_rn(q01, make_float2(m4.x, m4.y), beta2);
    beta2 = __ffma2_rn(q23, make_float2(m4.z, m4.w), beta2);
    // 2-bit: the odd slice of a word comes out 16 times larger
    const float f = BITS == 2 && (kk & 1) ? 0.0625f : 1.0f;
    const float2 x01 = __fmul2_rn(q01, make_float2(s4.x * f, s4.y * f)), x23 = __fmul2_rn(q23, make_float2(s4.z * f, s4.w * f));
    const __half2 h01 = __floats2half2_rn(x01.x, x01.y), h23 = __floats2half2_rn(x23.x, x23.y);
    const float2 r01 = __half22float2(h01), r23 = __half22float2(h23);
    const uint32_t a[4] = {*reinterpret_cast<const uint32_t*>(&h01), pack_f16x2(x01.x - r01.x, x01.y - r01.y),
                           *reinterpret_cast<const uint32_t*>(&h23), pack_f16x2(x23.x - r23.x, x23.y - r23.y)};
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      uint32_t k[4];
      if constexpr (BITS == 4) unpack8_sub(w[p][kk], k);
      else unpack_crumbs_sub(w[p][kk >> 1], kk & 1, k);
      mma16816(c[2 * p], a, k[0], k[2]);
      mma16816(c[2 * p + 1], a, k[1], k[3]);
    }
  }
  float beta = beta2.x + beta2.y;
  beta += __shfl_xor_sync(0xffffffffu, beta, 1);
  beta += __shfl_xor_sync(0xffffffffu, beta, 2);
  beta *= scale;
  const float lo = scale * kLowRows, hi = scale * (BITS == 4 ? kHighRows : 4194304.0f);
  float z[2][4];   // page p: tokens 2ti, 2ti+1, 2ti+8, 2ti+9 of column gi
#pragma unroll
  for (int p = 0; p < 2; ++p)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      z[p][e] = fmaf(c[2 * p][e] + c[2 * p][2 + e], lo, beta);
      z[p][2 + e] = fmaf(c[2 * p + 1][e] + c[2 * p + 1][2 + e], hi, beta);
    }
  if constexpr (SC) {
#pragma unroll
    for (int p = 0; p < 2; ++p)
      through_form(z[p], args, slope2, rel - 16 * p - 2 * ti, lane_token);
  }
  float mx = fmaxf(fmaxf(fmaxf(z[0][0], z[0][1]), fmaxf(z[0][2], z[0][3])), fmaxf(fmaxf(z[1][0], z[1][1]), fmaxf(z[1][2], z[1][3])));
  if (__any_sync(0xffffffffu, mx > m + kLazy)) {
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    const float mn = fmaxf(m, mx), al = mn == -INFINITY ? 1.0f : ex2(m - mn);
    m = mn;
    l *= al;
    const float a0 = __shfl_sync(0xffffffffu, al, 8 * ti), a1 = __shfl_sync(0xffffffffu, al, 8 * ti + 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      s.o[i][0] *= a0;
      s.o[i][1] *= a1;
      s.o[i][2] *= a0;
      s.o[i][3] *= a1;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) s.bias[k] *= al;
  }
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const char* rec = stage + p * RS;
#pragma unroll
    for (int x = 0; x < 4; ++x) z[p][x] = ex2(z[p][x] - m);
    l += (z[p][0] + z[p][1]) + (z[p][2] + z[p][3]);
    const float2 p01 = make_float2(z[p][0], z[p][1]), p23 = make_float2(z[p][2], z[p][3]);
    uint32_t b0[4], b1[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float4 s4 = *reinterpret_cast<const float4*>(rec + F::kVm + ((2 * k) * 4 + ti) * 16);
      const float4 m4 = *reinterpret_cast<const float4*>(rec + F::kVm + ((2 * k + 1) * 4 + ti) * 16);
      const float2 y01 = __fmul2_rn(p01, make_float2(s4.x, s4.y)), y23 = __fmul2_rn(p23, make_float2(s4.z, s4.w));
      b0[k] = pack_f16x2(y01.x, y01.y);
      b1[k] = pack_f16x2(y23.x, y23.y);
      float2 u = __ffma2_rn(p01, make_float2(m4.x, m4.y), make_float2(s.bias[k], 0.0f));
      u = __ffma2_rn(p23, make_float2(m4.z, m4.w), u);
      s.bias[k] = u.x + u.y;
    }
    uint32_t v[8];
    {
      const uint4 x = *reinterpret_cast<const uint4*>(rec + F::kVc + lane * 16);
      v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
      if constexpr (BITS == 4) {
        const uint4 y = *reinterpret_cast<const uint4*>(rec + F::kVc + 512 + lane * 16);
        v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
      }
    }
#pragma unroll
    for (int mt = 0; mt < 8; ++mt) {
      uint32_t a[4];
      if constexpr (BITS == 4) unpack8_sub(v[mt], a);
      else unpack_crumbs_sub(v[mt >> 1], mt & 1, a);
      mma16816(s.o[mt], a, b0[mt >> 1], b1[mt >> 1]);
    }
  }
  __syncwarp();   // the stage is read
}

// ---- KIVI pages: a block that is cut, or that the residual reaches into ------------------
// As the decode kernel's tail: keys from the staged records (whole groups) or the
// key-ring rows at `kring`, values below Tv from the records, later ones from the
// value-ring rows staged token-major at vrows. pos0, pos1: positions of columns
// 2ti and 2ti + 1.
template <int BITS, bool SC>
__device__ void kivi_cut_block(const Args<SC>& args, const Seg& sg, MmaState& s, float* ptile, const float (&q)[32],
                               const char* recs, const uint16_t* kring, const char* vrows, uint32_t zero_s, float scale,
                               const float* slope2, const Cut& cut, int pos0, int pos1) {
  using F = Rec<BITS>;
  constexpr int RS = kRecStrideB<BITS>;
  const int lane = threadIdx.x & 31, gi = lane >> 2, ti = lane & 3;
  const int t0 = cut.tok0, n = min(kG, sg.T - t0), t1 = t0 + n;
  float acc0[4] = {0.0f, 0.0f, 0.0f, 0.0f}, acc1[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  float beta = 0.0f;
  if (t0 + kG <= sg.Tk) beta = kscores_quant<true, BITS>(recs, q, acc0, acc1, kLoAbove / scale);
  else kscores_ring(kring, n, q, sg.dtype, acc0, acc1);
  const float bs0 = __shfl_sync(0xffffffffu, beta, 8 * ti) * scale, bs1 = __shfl_sync(0xffffffffu, beta, 8 * ti + 4) * scale;
  float z[8];   // tokens gi, gi + 8, 16 + gi, 24 + gi of columns 2ti (even entries) and 2ti + 1
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const float* acc = p ? acc1 : acc0;
    const int ta = t0 + 16 * p + gi, tb = ta + 8;
    if constexpr (SC) {
      const bool a0 = visible<SC>(ta, pos0, cut), a1 = visible<SC>(ta, pos1, cut), b0 = visible<SC>(tb, pos0, cut), b1 = visible<SC>(tb, pos1, cut);
      // (a masked score has no say in how the others are capped)
      float y0[2] = {a0 ? fmaf(acc[0], scale, bs0) : 0.0f, b0 ? fmaf(acc[2], scale, bs0) : 0.0f};
      float y1[2] = {a1 ? fmaf(acc[1], scale, bs1) : 0.0f, b1 ? fmaf(acc[3], scale, bs1) : 0.0f};
      auto on = [](int x) { return 8.0f * x; };
      through_form(y0, args, slope2[2 * ti * kPRow], pos0 - ta, on);
      through_form(y1, args, slope2[(2 * ti + 1) * kPRow], pos1 - ta, on);
      z[4 * p + 0] = a0 ? y0[0] : -INFINITY;
      z[4 * p + 1] = a1 ? y1[0] : -INFINITY;
      z[4 * p + 2] = b0 ? y0[1] : -INFINITY;
      z[4 * p + 3] = b1 ? y1[1] : -INFINITY;
    } else {
      z[4 * p + 0] = visible<SC>(ta, pos0, cut) ? fmaf(acc[0], scale, bs0) : -INFINITY;
      z[4 * p + 1] = visible<SC>(ta, pos1, cut) ? fmaf(acc[1], scale, bs1) : -INFINITY;
      z[4 * p + 2] = visible<SC>(tb, pos0, cut) ? fmaf(acc[2], scale, bs0) : -INFINITY;
      z[4 * p + 3] = visible<SC>(tb, pos1, cut) ? fmaf(acc[3], scale, bs1) : -INFINITY;
    }
  }
  float mx0 = fmaxf(fmaxf(z[0], z[2]), fmaxf(z[4], z[6])), mx1 = fmaxf(fmaxf(z[1], z[3]), fmaxf(z[5], z[7]));
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) {
    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o));
    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o));
  }
  if (__any_sync(0xffffffffu, mx0 > s.m0 + kLazy || mx1 > s.m1 + kLazy)) {
    const float mn0 = fmaxf(s.m0, mx0), mn1 = fmaxf(s.m1, mx1);
    const float al0 = mn0 == -INFINITY ? 1.0f : ex2(s.m0 - mn0), al1 = mn1 == -INFINITY ? 1.0f : ex2(s.m1 - mn1);
    s.m0 = mn0;
    s.m1 = mn1;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      s.o[i][0] *= al0;
      s.o[i][1] *= al1;
      s.o[i][2] *= al0;
      s.o[i][3] *= al1;
    }
    s.l0 *= al0;
    s.l1 *= al1;
    // bias belongs to column gi: its factor sits in lanes with ti = gi / 2
    const float a_even = __shfl_sync(0xffffffffu, al0, gi >> 1), a_odd = __shfl_sync(0xffffffffu, al1, gi >> 1);
#pragma unroll
    for (int k = 0; k < 4; ++k) s.bias[k] *= (gi & 1) ? a_odd : a_even;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] = z[i] == -INFINITY ? 0.0f : ex2(z[i] - ((i & 1) ? s.m1 : s.m0));
  s.l0 += (z[0] + z[2]) + (z[4] + z[6]);
  s.l1 += (z[1] + z[3]) + (z[5] + z[7]);
#pragma unroll
  for (int r = 0; r < 4; ++r) *reinterpret_cast<float2*>(ptile + (8 * r + gi) * kPRow + 2 * ti) = make_float2(z[2 * r], z[2 * r + 1]);
  __syncwarp();
  const int vt0 = max(t0, sg.Tv);
  // a value-ring row that only some columns see and that is not finite (lane = row)
  bool wildrow = false;
  if (cut.first != cut.last && lane < n && t0 + lane >= vt0) {
    const uint4* row = reinterpret_cast<const uint4*>(vrows + lane * kVRow);
    for (int c = 0; c < 16; ++c) {
      const uint4 w = row[c];
      if (sg.dtype == S4KV_BF16)
        wildrow = wildrow || wild<S4KV_BF16>(w.x) || wild<S4KV_BF16>(w.y) || wild<S4KV_BF16>(w.z) || wild<S4KV_BF16>(w.w);
      else
        wildrow = wildrow || wild<S4KV_F16>(w.x) || wild<S4KV_F16>(w.y) || wild<S4KV_F16>(w.z) || wild<S4KV_F16>(w.w);
    }
  }
  const bool apart = __any_sync(0xffffffffu, wildrow);
#pragma unroll 1
  for (int p = 0; p < 2; ++p) {
    const int tb = t0 + 16 * p;
    if (tb >= t1) break;
    // p of tokens 2ti, 2ti+1, 2ti+8, 2ti+9 of this page, column gi
    float pe[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) pe[x] = ptile[(16 * p + 2 * ti + (x & 1) + 8 * (x >> 1)) * kPRow + gi];
    if (tb < sg.Tv) {   // restored values: tokens tb .. Tv - 1 of this page
      const char* rec = recs + p * RS;
      const int nq = sg.Tv - tb;
      bool on[4];       // masked tokens (p = 0) stay out: their scale may be anything
#pragma unroll
      for (int x = 0; x < 4; ++x) on[x] = 2 * ti + (x & 1) + 8 * (x >> 1) < nq && pe[x] > 0.0f;
      uint32_t b0[4], b1[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 s4 = *reinterpret_cast<const float4*>(rec + F::kVm + ((2 * k) * 4 + ti) * 16);
        const float4 m4 = *reinterpret_cast<const float4*>(rec + F::kVm + ((2 * k + 1) * 4 + ti) * 16);
        b0[k] = pack_f16x2(on[0] ? pe[0] * s4.x : 0.0f, on[1] ? pe[1] * s4.y : 0.0f);
        b1[k] = pack_f16x2(on[2] ? pe[2] * s4.z : 0.0f, on[3] ? pe[3] * s4.w : 0.0f);
        float bk = s.bias[k];
        bk = on[0] ? fmaf(pe[0], m4.x, bk) : bk;
        bk = on[1] ? fmaf(pe[1], m4.y, bk) : bk;
        bk = on[2] ? fmaf(pe[2], m4.z, bk) : bk;
        bk = on[3] ? fmaf(pe[3], m4.w, bk) : bk;
        s.bias[k] = bk;
      }
      uint32_t vd[8];
      {
        const uint4 v0 = *reinterpret_cast<const uint4*>(rec + F::kVc + lane * 16);
        vd[0] = v0.x; vd[1] = v0.y; vd[2] = v0.z; vd[3] = v0.w;
        if constexpr (BITS == 4) {
          const uint4 v1 = *reinterpret_cast<const uint4*>(rec + F::kVc + 512 + lane * 16);
          vd[4] = v1.x; vd[5] = v1.y; vd[6] = v1.z; vd[7] = v1.w;
        }
      }
#pragma unroll
      for (int mt = 0; mt < 8; ++mt) {
        uint32_t a[4];
        if constexpr (BITS == 4) unpack8(vd[mt], a);
        else unpack_crumbs(vd[mt >> 1], mt & 1, a);
        mma16816(s.o[mt], a, b0[mt >> 1], b1[mt >> 1]);
      }
    }
    if (tb + kP > vt0) {   // value-ring rows of this page
      // this lane's ldmatrix row: matrix j = lane / 8 (tokens + 8 for j >= 2,
      // channels + 8 for odd j), row lane % 8
      const int j = lane >> 3;
      const int row = 16 * p + (lane & 7) + 8 * (j >> 1), t = t0 + row;
      const bool there = t >= vt0 && t < t1;
      const int opos[2] = {pos0, pos1};
      auto pv = [&](bool present, const float (&y)[4], int only) {   // only: as in byte_block
        const uint32_t base = present ? smem_u32(vrows + row * kVRow + 16 * (j & 1)) : zero_s;
        const uint32_t step = present ? 32u : 0u;   // 16 channels further per tile
        if (sg.dtype == S4KV_BF16) {
          const uint32_t h0 = pack_bf16x2(y[0], y[1]), h1 = pack_bf16x2(y[2], y[3]);
          const uint32_t l0 = pack_bf16x2(y[0] - __uint_as_float(h0 << 16), y[1] - __uint_as_float(h0 & 0xffff0000u));
          const uint32_t l1 = pack_bf16x2(y[2] - __uint_as_float(h1 << 16), y[3] - __uint_as_float(h1 & 0xffff0000u));
#pragma unroll
          for (int mt = 0; mt < 8; ++mt) {
            uint32_t a[4];
            ldsm_x4_trans(base + mt * step, a);
            auto product = [&](float (&t)[4]) {
              mma16816_bf16(t, a, h0, h1);
              mma16816_bf16(t, a, l0, l1);
            };
            if (only < 0) product(s.o[mt]);
            else add_only(s.o[mt], opos, only, product);
          }
        } else {
          const uint32_t h0 = pack_f16x2(y[0], y[1]), h1 = pack_f16x2(y[2], y[3]);
          const float2 f0 = unpack_in<S4KV_F16>(h0), f1 = unpack_in<S4KV_F16>(h1);
          const uint32_t l0 = pack_f16x2(y[0] - f0.x, y[1] - f0.y), l1 = pack_f16x2(y[2] - f1.x, y[3] - f1.y);
#pragma unroll
          for (int mt = 0; mt < 8; ++mt) {
            uint32_t a[4];
            ldsm_x4_trans(base + mt * step, a);
            auto product = [&](float (&t)[4]) {
              mma16816(t, a, h0, h1);
              mma16816(t, a, l0, l1);
            };
            if (only < 0) product(s.o[mt]);
            else add_only(s.o[mt], opos, only, product);
          }
        }
      };
      // quantized tokens of this page already entered through their records
      float y[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) y[x] = tb + 2 * ti + (x & 1) + 8 * (x >> 1) >= vt0 ? pe[x] : 0.0f;
      if (!apart) {
        pv(there && visible_to<SC>(t, cut.first, cut.last, cut), y, -1);
      } else {
        for (int qp = cut.first; qp <= cut.last; ++qp) pv(there && visible<SC>(t, qp, cut), y, qp);
      }
    }
  }
  __syncwarp();
}

// ---- the kernel ----------------------------------------------------------------------------
__device__ __forceinline__ long long* win_meta(const WindowArgs& a) {
  return reinterpret_cast<long long*>(a.ws + 2LL * a.grid_warps * partial_floats(a.pcols));
}

// Eight consecutive channels from c on of one output row.
__device__ __forceinline__ void store8(const WindowArgs& a, long long row, int c, const float (&y)[8]) {
  const long long idx = row * kD + c;
  if (a.out_dtype == S4KV_F32) {
    float4* p = reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + idx);
    p[0] = make_float4(y[0], y[1], y[2], y[3]);
    p[1] = make_float4(y[4], y[5], y[6], y[7]);
  } else {
    uint4 w;
    w.x = pack_in_dtype(y[0], y[1], a.out_dtype);
    w.y = pack_in_dtype(y[2], y[3], a.out_dtype);
    w.z = pack_in_dtype(y[4], y[5], a.out_dtype);
    w.w = pack_in_dtype(y[6], y[7], a.out_dtype);
    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.out) + idx) = w;
  }
}
__device__ __forceinline__ void store1(const WindowArgs& a, long long row, int c, float y) {
  const long long idx = row * kD + c;
  if (a.out_dtype == S4KV_F32) reinterpret_cast<float*>(a.out)[idx] = y;
  else if (a.out_dtype == S4KV_BF16) reinterpret_cast<__nv_bfloat16*>(a.out)[idx] = __float2bfloat16_rn(y);
  else reinterpret_cast<__half*>(a.out)[idx] = __float2half_rn(y);
}

// The combine of a one-segment launch: a cluster's CTAs hold one segment, each warp
// left its columns' (m, l) in wm, wl and its unscaled output in its region. First the
// warps of a CTA (a thread per four channels of a column), then, column by column,
// the CTAs through distributed shared memory. Warps without work left l = 0 and
// nothing else. Every thread of the cluster comes here once.
template <int FMT, int NC, bool SC>
__device__ __forceinline__ void combine_cluster(const WindowArgs& a, const WSmem<FMT, NC, SC>& sm, OneSmem& one, int csize, int rank, int ncols,
                                                long long row0, int col0, int g) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // output row of the tile's column j
  auto out_row = [&](int j) -> long long {
    const int i = (col0 + j) / g;
    return row0 + static_cast<long long>(i) * a.Hq + (col0 + j - i * g);
  };
  auto finish = [&](int col, float L, float4 O) {
    const float inv = L > 0.0f ? 1.0f / L : L == L ? 0.0f : L;
    store_out(a, out_row(col), lane, make_float4(O.x * inv, O.y * inv, O.z * inv, O.w * inv));
  };
  __syncthreads();
  for (int col = warp; col < ncols; col += kWarps) {
    float M = -INFINITY, L = 0.0f;
    float4 O = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, one.wm[w][col]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float l = one.wl[w][col];
      if (l == 0.0f) continue;
      const float x = M == -INFINITY ? 1.0f : ex2(one.wm[w][col] - M);
      const float4 r = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(sm.region[w]) + col * kD + 4 * lane);
      L = fmaf(x, l, L);
      O = make_float4(fmaf(x, r.x, O.x), fmaf(x, r.y, O.y), fmaf(x, r.z, O.z), fmaf(x, r.w, O.w));
    }
    if (csize == 1) {
      finish(col, L, O);
    } else {
      *reinterpret_cast<float4*>(&one.part[col][4 * lane]) = O;
      if (lane == 0) {
        one.pm[col] = M;
        one.pl[col] = L;
      }
    }
  }
  if (csize == 1) return;
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  auto remote = [&](const void* p, int r) {
    uint32_t x;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(x) : "r"(smem_u32(p)), "r"(r));
    return x;
  };
  for (int col = warp * csize + rank; col < ncols; col += kWarps * csize) {
    float M = -INFINITY, L = 0.0f, m = -INFINITY, l = 0.0f;
    float4 O = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (lane < csize) {
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(m) : "r"(remote(&one.pm[col], lane)));
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(l) : "r"(remote(&one.pl[col], lane)));
    }
    M = warp_max(m);
    const float wl = l == 0.0f ? 0.0f : M == -INFINITY ? 1.0f : ex2(m - M);
    for (int r = 0; r < csize; ++r) {
      const float x = __shfl_sync(0xffffffffu, wl, r), lr = __shfl_sync(0xffffffffu, l, r);
      if (lr == 0.0f) continue;
      float4 y;
      asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(y.x), "=f"(y.y), "=f"(y.z), "=f"(y.w)
                   : "r"(remote(&one.part[col][4 * lane], r)));
      L = fmaf(x, lr, L);
      O = make_float4(fmaf(x, y.x, O.x), fmaf(x, y.y, O.y), fmaf(x, y.z, O.z), fmaf(x, y.w, O.w));
    }
    finish(col, L, O);
  }
  // no CTA leaves while another may still read its shared memory
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// x / y, x >= 0 and y > 0, in 32 bits where they do (a 64-bit division takes several hundred cycles).
__device__ __forceinline__ long long quotient(long long x, long long y) {
  return (x | y) >> 32 ? x / y : static_cast<unsigned>(x) / static_cast<unsigned>(y);
}
// Where part i of n parts of C starts.
__device__ __forceinline__ long long part_of(long long C, int i, int n) { return quotient(i * C, n); }

// FMT: page format. NC: columns a warp holds (8, or 16 on 8-bit pages).
// ONE: a cluster of CTAs holds one segment and combines it itself (grid.x = CTAs of
// a cluster, grid.y = segments); otherwise the slices of the whole line, as above.
template <int FMT, int NC, bool ONE, bool SC>
__global__ void __launch_bounds__(32 * kWarps, 1) window_kernel(Args<SC> a) {
  constexpr int BT = kBlock<FMT>;
  constexpr int CT = NC / 8;
  constexpr int kThreads = 32 * kWarps;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  auto& sm = *reinterpret_cast<WSmem<FMT, NC, SC>*>(smem_raw);
  long long* pre = reinterpret_cast<long long*>(smem_raw + prefix_at<FMT, NC, SC>());   // [B + 1]
  OneSmem& one = *reinterpret_cast<OneSmem*>(smem_raw + prefix_at<FMT, NC, SC>());        // (ONE)
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gi = lane >> 2, ti = lane & 3;
  uint8_t* region = sm.region[warp];
  uint64_t* bar = sm.bar[warp];
  if (lane == 0)
    for (int i = 0; i < 4; ++i) mbar_init(&bar[i], 1);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  __shared__ __align__(16) uint4 zero16;
  if (tid == 0) zero16 = make_uint4(0u, 0u, 0u, 0u);
  stream_wait();
  int b, seg, T, gw, n_act;
  long long r0, r1, seg_start, C = 0;
  Plan<FMT> pl;
  Span own_span;   // of query `lane` of sequence b
  if constexpr (ONE) {
    const int per = a.H * a.tiles;
    b = static_cast<int>(blockIdx.y) / per;
    seg = static_cast<int>(blockIdx.y) - b * per;
    T = a.seq_lens[b];
    pl = plan_of_warp<FMT, SC>(T, a, b, own_span);
    gw = warp * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x);
    n_act = static_cast<int>(gridDim.x) * kWarps;
    if (a.max_warps > 0 && a.max_warps < n_act) n_act = a.max_warps;
    if (pl.work < n_act) n_act = static_cast<int>(pl.work);
    seg_start = 0;
    r0 = part_of(pl.work, gw, n_act);
    r1 = part_of(pl.work, gw + 1, n_act);
    if (gw >= n_act) r1 = 0;
    if (lane < NC) {
      one.wm[warp][lane] = -INFINITY;
      one.wl[warp][lane] = 0.0f;
    }
    __syncthreads();
  } else {
    {   // cost prefix over sequences: sequence b owns H tiles segments of its plan's cost
      long long carry = 0;
      __shared__ long long wt[kWarps];
      for (int base = 0; base < a.B; base += kThreads) {
        const int b = base + tid;
        const long long cnt = b < a.B ? static_cast<long long>(a.H) * a.tiles * plan_of<FMT, SC>(a.seq_lens[b], a, b).cost() : 0;
        long long x = cnt;
  #pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        if (lane == 31) wt[warp] = x;
        __syncthreads();
        long long before = carry, total = 0;
        for (int q = 0; q < kWarps; ++q) {
          if (q < warp) before += wt[q];
          total += wt[q];
        }
        if (b < a.B) pre[b] = before + x - cnt;
        __syncthreads();
        carry += total;
      }
      if (tid == 0) pre[a.B] = carry;
      __syncthreads();
    }
    C = pre[a.B];
    n_act = static_cast<int>(gridDim.x) * kWarps;
    if (a.max_warps > 0 && a.max_warps < n_act) n_act = a.max_warps;
    {
      const long long cap = (C + kLeastUnits<FMT> - 1) / kLeastUnits<FMT>;
      if (cap < n_act) n_act = static_cast<int>(cap);
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    gw = warp * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x);
    if (gw >= n_act) return;
    r0 = part_of(C, gw, n_act);
    r1 = part_of(C, gw + 1, n_act);
    {   // first sequence touching this slice
      int lo = 0, hi = a.B - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (pre[mid] <= r0) lo = mid; else hi = mid - 1;
      }
      b = lo;
    }
    T = a.seq_lens[b];
    pl = plan_of_warp<FMT, SC>(T, a, b, own_span);
    seg = static_cast<int>(quotient(r0 - pre[b], pl.cost()));   // h * tiles + tile, within the sequence
    seg_start = pre[b] + seg * pl.cost();
    if (kSegCost<FMT> > 0 && r0 - seg_start >= pl.work) {   // nothing of this segment is left
      seg_start += pl.cost();
      if (++seg == a.H * a.tiles) {
        seg = 0;
        if (++b >= a.B) return;
        T = a.seq_lens[b];
        pl = plan_of_warp<FMT, SC>(T, a, b, own_span);
      }
    }
  }

  uint32_t phase = 0, pend = 0;   // per-stage wait parity and copies in flight (bit per stage)
  const uint64_t once = policy_evict_first();
  bool aborted = false;
  auto wait = [&](int s) -> bool {
    if (!mbar_wait(&bar[s], (phase >> s) & 1u, aborted ? 0 : a.wait_ns)) return false;
    phase ^= 1u << s;
    pend &= ~(1u << s);
    return true;
  };
  auto fail = [&](int where) {   // a bounded wait ran out: drain, then go on without compute
    if (lane == 0) report(a.status, S4KV_ERR_DEVICE_TIMEOUT, S4KV_DEV_TIMEOUT, where);
    aborted = true;
    for (int s = 0; s < 4; ++s)
      if ((pend >> s) & 1u) {
        mbar_wait(&bar[s], (phase >> s) & 1u, kDrainNs);
        phase ^= 1u << s;
        pend &= ~(1u << s);
      }
  };

  const int ncols = a.nq * a.g, by_g = 65536 / a.g + 1;   // col / g = col by_g >> 16: col g < 65536

  while (seg_start < r1) {
    const long long seg_end = seg_start + pl.work;   // of its blocks
    const long long lo = max(r0, seg_start) - seg_start, hi = min(r1, seg_end) - seg_start;
    const bool own = !ONE && lo == 0 && hi == pl.work;
    const int h = seg / a.tiles, col0 = (seg - h * a.tiles) * NC;
    const int slot = a.slot_ids ? a.slot_ids[b] : b;
    const bool slot_ok = slot >= 0 && slot < a.max_slots;
    // what the segment needs from memory, all of it on its way at once: the stored length, the column's slope,
    // the pages of its first units and (8-bit pages) the queries
    const bool shape_ok = T > 0 && T >= a.nq && T <= a.max_seq_len && static_cast<long long>(a.bt_stride) * kP >= T;
    const int lens_v = slot_ok ? __ldcg(a.lens + slot * a.H + h) : 0;
    // positions: of a column past the last one, the last query's
    auto pos_of = [&](int col) { return T - a.nq + (min(col, ncols - 1) * by_g >> 16); };
    auto qrow_of = [&](int col) -> const uint16_t* {
      if (col >= ncols) return nullptr;
      const int i = col * by_g >> 16;
      return a.q + ((static_cast<long long>(b) * a.nq + i) * a.Hq + h * a.g + (col - i * a.g)) * kD;
    };
    auto out_row = [&](int col) -> long long {
      const int i = col * by_g >> 16;
      return (static_cast<long long>(b) * a.nq + i) * a.Hq + h * a.g + (col - i * a.g);
    };
    float slope = 0.0f;   // of column `lane`
    if constexpr (SC) {
      if (lane < NC && a.score.slopes && col0 + lane < ncols) slope = a.score.slopes[h * a.g + col0 + lane - ((col0 + lane) * by_g >> 16) * a.g] * 1.4426950408889634f;
    }
    const int* bt = a.block_table + static_cast<long long>(b) * a.bt_stride;
    int u0 = 0, u1 = 0, n = 0, first_pp = 0;   // (8-bit pages)
    bool ring = false;
    constexpr bool kEarly = FMT == kI8 || NC == 16;   // (FP8, 8 columns: 2% slower with them early)
    uint4 qrows[CT][4];
    const uint16_t* qrow[CT];
    auto fetch_q = [&](int c) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        qrows[c][j] = qrow[c] ? reinterpret_cast<const uint4*>(qrow[c])[4 * ti + j] : make_uint4(0u, 0u, 0u, 0u);
    };
    if constexpr (kByte<FMT>) {
      const int units = pl.nf + pl.nx;   // the last one may be the unfinished block, of more than one position
      u0 = min(static_cast<int>(lo), units);
      u1 = min(static_cast<int>(hi), units);
      ring = FMT == kI8 && (T % kP) != 0 && u0 < u1 && u1 == units;
      n = u1 - u0 - (ring ? 1 : 0);                                  // records to stream
      if (shape_ok && lane < n) first_pp = bt[pl.block_of(u0 + lane)];
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        qrow[c] = qrow_of(col0 + 8 * c + gi);
        if (kEarly) fetch_q(c);
      }
    }
    Cut cut;
    cut.tok0 = 0;
    cut.window = a.window;
    cut.sinks = a.sinks;
    cut.first = pos_of(col0);
    cut.last = pos_of(min(col0 + NC, ncols) - 1);
    if constexpr (SC) {
      float* spans = kByte<FMT> ? reinterpret_cast<float*>(sm.spans[kByte<FMT> ? warp : 0]) : sm.ptile[kByte<FMT> ? 0 : warp] + kSpanAt;
      float* slopes = kByte<FMT> ? sm.slope2[kByte<FMT> ? warp : 0] : sm.ptile[kByte<FMT> ? 0 : warp] + kSlopeAt;
      constexpr int kEach = kByte<FMT> ? 1 : kPRow;
      cut.step = kByte<FMT> ? 2 : kPRow;
      cut.spans = spans;
      cut.base = T - a.nq;
      __syncwarp();   // the segment before is done with its spans
      Span mine{0x7fffffff, -1};
      if (lane < a.nq && T > 0) {
        const int p = T - a.nq + lane;
        *reinterpret_cast<Span*>(spans + lane * cut.step) = own_span;
        if (p >= cut.first && p <= cut.last) mine = own_span;
      }
      if (lane < NC) slopes[lane * kEach] = slope;
      cut.lo = __reduce_min_sync(0xffffffffu, mine.lo);
      cut.hi = __reduce_max_sync(0xffffffffu, mine.hi);
      __syncwarp();
    }
    bool valid = slot_ok && T > 0;
    if (!slot_ok) {
      if (lane == 0) report(a.status, S4KV_ERR_DEVICE, S4KV_DEV_BAD_SLOT, slot);
    } else if (lens_v != T || T > a.max_seq_len || (T > 0 && T < a.nq)) {
      valid = false;
      if (lane == 0) report(a.status, S4KV_ERR_DEVICE, S4KV_DEV_BAD_LENGTH, b);
    } else if (static_cast<long long>(a.bt_stride) * kP < T) {
      valid = false;
      if (lane == 0) report(a.status, S4KV_ERR_DEVICE, S4KV_DEV_BAD_TABLE, b);
    }
    valid = valid && !aborted;
    auto in_pool = [&](int pp) -> int {   // a pool page, -1 (reported) if outside the pool
      if (pp >= 0 && pp < a.num_pages) return pp;
      report(a.status, S4KV_ERR_DEVICE, S4KV_DEV_BAD_PAGE, pp);
      return -1;
    };
    auto page = [&](int lp) -> int { return in_pool(bt[lp]); };   // of logical page lp
    const uint16_t* kring = reinterpret_cast<const uint16_t*>(a.kring) + (slot_ok ? slot : 0) * a.kring_slot + h * a.kring_head;
    const uint16_t* vring = reinterpret_cast<const uint16_t*>(a.vring) + (slot_ok ? slot : 0) * a.vring_slot + h * a.vring_head;

    if constexpr (kByte<FMT>) {
      ByteState<NC> st;
      byte_init(st);
      if (valid) {
        auto pages_of = [&](int k) -> int {   // pool pages of units u0 + 32 k + lane
          const int x = 32 * k + lane;
          return x < n ? page(pl.block_of(u0 + x)) : 0;
        };
        int curp = lane < n ? in_pool(first_pp) : 0, nxtp = n > 32 ? pages_of(1) : 0, cur_k = 0;
        int pos[CT], opos[CT][2];
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          pos[c] = pos_of(col0 + 8 * c + gi);
          opos[c][0] = pos_of(col0 + 8 * c + 2 * ti);
          opos[c][1] = pos_of(col0 + 8 * c + 2 * ti + 1);
        }
        uint32_t skip = 0;
        auto issue = [&](int s, int i) {   // i = 0, 1, 2, ... in order
          if ((i >> 5) != cur_k) {
            curp = nxtp;
            ++cur_k;
            nxtp = pages_of(cur_k + 1);
          }
          const int pp = __shfl_sync(0xffffffffu, curp, i & 31);
          if (pp < 0) {
            skip |= 1u << s;
            return;
          }
          skip &= ~(1u << s);
          constexpr uint32_t kCopy = FMT == kI8 ? Rec<kI8>::kCopy : Rec<8>::kBytes;
          fence_proxy_async();   // earlier generic reads of the stage come first
          __syncwarp();
          if (lane == 0) {
            const char* src = a.pages + (static_cast<long long>(pp) * a.H + h) * Rec<FMT>::kBytes;
            mbar_expect_tx(&bar[s], kCopy);
            bulk_load_hint(region + s * Rec<kI8>::kBytes, src, kCopy, &bar[s], once);
          }
          pend |= 1u << s;
        };
        for (int i = 0; i < n && i < kStagesOf<FMT>; ++i) issue(i, i);
        // queries: f16 operands, and (INT8) -128 scale sum_c q_c
        const float ks = FMT == 8 ? a.fp8_scale[h] : 0.0f;
        uint32_t qa[8][2];        // 8 columns: row gi, channels c_0 c_1 | c_2 c_3 of slice kk
        float zoff[CT], zscale0 = 0.0f;
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          if (!kEarly) fetch_q(c);
          const uint4 (&row)[4] = qrows[c];
          float up = 1.0f;
          float zscale = a.sm_scale_log2 * (FMT == kI8 ? 16777216.0f : ks);
          if (a.dtype == S4KV_BF16) {
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              top = __vmaxu2(__vmaxu2(__vmaxu2(__vmaxu2(top, row[j].x & 0x7fff7fffu), row[j].y & 0x7fff7fffu), row[j].z & 0x7fff7fffu),
                             row[j].w & 0x7fff7fffu);
            top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int k = query_power(max(top & 0xffffu, top >> 16));
            up = power_of_two(k);
            zscale *= power_of_two(-k);
          }
          zscale0 = zscale;   // (8 columns)
          if (NC == 16 && ti == 0) sm.zscale[warp][8 * c + gi] = zscale;
          float sum = 0.0f;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t w[4] = {row[j].x, row[j].y, row[j].z, row[j].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t x = w[i];
              if (a.dtype == S4KV_BF16)
                x = pack_f16x2(__uint_as_float(x << 16) * up, __uint_as_float(x & 0xffff0000u) * up);
              if constexpr (NC == 8) qa[2 * j + (i >> 1)][i & 1] = x;
              else reinterpret_cast<uint32_t*>(&sm.q[warp][2 * j + (i >> 1)][lane])[2 * (i & 1) + c] = x;
              if (FMT == kI8) {
                const float2 f = unpack_in<S4KV_F16>(x);
                sum += f.x + f.y;
              }
            }
          }
          sum += __shfl_xor_sync(0xffffffffu, sum, 1);
          sum += __shfl_xor_sync(0xffffffffu, sum, 2);
          zoff[c] = -128.0f / 16777216.0f * zscale * sum;
        }
        if (NC == 16) __syncwarp();   // the columns' scales are there
        bool ok = true;
        int s = 0;
        for (int i = 0; i < n; ++i) {
          if (!((skip >> s) & 1u)) {
            if (!wait(s)) {
              ok = false;
              break;
            }
            const char* rec = reinterpret_cast<const char*>(region + s * Rec<kI8>::kBytes);
            if (SC || u0 + i >= pl.nf) cut.tok0 = pl.block_of(u0 + i) * BT;
            const float* slopes = sm.slope2[SC ? warp : 0];
            if (u0 + i < pl.nf)
              byte_block<FMT, NC, false, SC>(a, rec, st, qa, sm.q[NC == 16 ? warp : 0], zoff, zscale0, sm.zscale[NC == 16 ? warp : 0], slopes, cut, pos, opos);
            else
              byte_block<FMT, NC, true, SC>(a, rec, st, qa, sm.q[NC == 16 ? warp : 0], zoff, zscale0, sm.zscale[NC == 16 ? warp : 0], slopes, cut, pos, opos);
          }
          if (i + kStagesOf<FMT> < n) issue(s, i + kStagesOf<FMT>);
          s = s + 1 == kStagesOf<FMT> ? 0 : s + 1;
        }
        {
          const float vs = FMT == 8 ? a.fp8_scale[a.H + h] : kI8Rest;
#pragma unroll
          for (int mt = 0; mt < 8; ++mt)
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
              for (int e = 0; e < 4; ++e) st.o[mt][c][e] *= vs;
        }
        if (ok && ring) {
          cut.tok0 = T / kP * kP;
          const float* slopes = sm.slope2[SC ? warp : 0];
          if (a.dtype == S4KV_BF16) ring_block<S4KV_BF16, NC, SC>(a, kring, vring, T % kP, st, qrow, a.sm_scale_log2, slopes, cut, pos, opos);
          else ring_block<S4KV_F16, NC, SC>(a, kring, vring, T % kP, st, qrow, a.sm_scale_log2, slopes, cut, pos, opos);
        }
        if (!ok) {
          fail(b);
          byte_init(st);
        }
      }
      // ---- output, or the partial that win_merge_kernel combines ----
      float f[CT][2];
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        st.l[c] += __shfl_xor_sync(0xffffffffu, st.l[c], 1);
        st.l[c] += __shfl_xor_sync(0xffffffffu, st.l[c], 2);
#pragma unroll
        for (int e = 0; e < 2; ++e) {   // columns 8c + 2ti + e: their sums sit in lanes 8ti + 4e
          const float l = __shfl_sync(0xffffffffu, st.l[c], 8 * ti + 4 * e);
          f[c][e] = own ? (l > 0.0f ? 1.0f / l : l == l ? 0.0f : l) : 1.0f;
        }
      }
      const bool direct = !ONE && (own || !slot_ok);
      const int k = seg_start <= r0 ? 0 : 1;
      float* P = ONE ? reinterpret_cast<float*>(region) : a.ws + (2LL * gw + k) * partial_floats(a.pcols);
      if constexpr (ONE) __syncwarp();   // the region's records are read
#pragma unroll
      for (int c = 0; c < CT; ++c) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int col = 8 * c + 2 * ti + e;
          if (col0 + col < ncols) {
            const long long row = out_row(col0 + col);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              float y[8];
#pragma unroll
              for (int mt = 0; mt < 8; ++mt) y[mt] = st.o[mt][c][2 * half + e] * f[c][e];
              if constexpr (FMT == kI8) {   // channels 64 half + 8 gi + mt
                if (direct) store8(a, row, 64 * half + 8 * gi, y);
                else {
                  float4* d = reinterpret_cast<float4*>(P + col * kD + 64 * half + 8 * gi);
                  d[0] = make_float4(y[0], y[1], y[2], y[3]);
                  d[1] = make_float4(y[4], y[5], y[6], y[7]);
                }
              } else {   // channels 16 mt + 8 half + gi
#pragma unroll
                for (int mt = 0; mt < 8; ++mt) {
                  if (direct) store1(a, row, 16 * mt + 8 * half + gi, y[mt]);
                  else P[col * kD + 16 * mt + 8 * half + gi] = y[mt];
                }
              }
            }
          }
        }
        if (ONE) {
          if (ti == 0) {
            one.wm[warp][8 * c + gi] = st.m[c];
            one.wl[warp][8 * c + gi] = st.l[c];
          }
        } else if (!direct && ti == 0 && col0 + 8 * c + gi < ncols) {
          P[a.pcols * kD + 2 * (8 * c + gi)] = st.m[c];
          P[a.pcols * kD + 2 * (8 * c + gi) + 1] = st.l[c];
        }
      }
    } else {
      using F = Rec<FMT>;
      constexpr int RS = kRecStrideB<FMT>;
      float* ptile = sm.ptile[warp];
      uint8_t* st0 = region;
      uint8_t* st1 = region + kStageBytesB<FMT>;
      MmaState ms;
      mma_init(ms);
      GenState gs;
      bool have = false;
      if (valid) {
        const int nf = pl.nf, tc = a.tail_cost;
        const int u0 = static_cast<int>(lo < nf ? lo : nf), u1 = static_cast<int>(hi < nf ? hi : nf), n = u1 - u0;
        int c0 = 0, c1 = 0;   // cut blocks whose cost position starts inside [lo, hi)
        if (pl.nx > 0 && hi > nf) {
          c0 = static_cast<int>(lo > nf ? (lo - nf + tc - 1) / tc : 0);
          const long long cc = (hi - nf + tc - 1) / tc;
          c1 = static_cast<int>(cc < pl.nx ? cc : pl.nx);
        }
        Seg sg;
        sg.pages = a.pages;
        sg.bt = bt;
        sg.kring = kring;
        sg.vring = vring;
        sg.H = a.H;
        sg.h = h;
        sg.T = T;
        sg.Tk = T & ~(kG - 1);
        sg.Tv = max(0, T - a.R);
        sg.R = a.R;
        sg.dtype = a.dtype;
        auto pages_of = [&](int k, int& x0, int& x1) {   // both pages of units u0 + 32 k + lane
          const int x = 32 * k + lane;
          x0 = x1 = 0;
          if (x < n) {
            const int blk = pl.block_of(u0 + x);
            x0 = page(2 * blk);
            x1 = page(2 * blk + 1);
            if (x1 < 0) x0 = -1;
          }
        };
        int cur0, cur1, nxt0 = 0, nxt1 = 0, cur_k = 0;
        pages_of(0, cur0, cur1);
        if (n > 32) pages_of(1, nxt0, nxt1);
        uint32_t skip = 0;
        auto issue = [&](int s, int i) {
          if ((i >> 5) != cur_k) {
            cur0 = nxt0;
            cur1 = nxt1;
            ++cur_k;
            pages_of(cur_k + 1, nxt0, nxt1);
          }
          const int p0 = __shfl_sync(0xffffffffu, cur0, i & 31), p1 = __shfl_sync(0xffffffffu, cur1, i & 31);
          if (p0 < 0) {
            skip |= 1u << s;
            return;
          }
          skip &= ~(1u << s);
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) {
            uint8_t* dst = s ? st1 : st0;
            mbar_expect_tx(&bar[s], 2 * F::kBytes);
            bulk_load_hint(dst, rec_at<FMT>(sg, p0), F::kBytes, &bar[s], once);
            bulk_load_hint(dst + RS, rec_at<FMT>(sg, p1), F::kBytes, &bar[s], once);
          }
          pend |= 1u << s;
        };
        for (int i = 0; i < n && i < kStages; ++i) issue(i, i);
        // this lane's query: column gi, channels 32 ti + x
        const uint16_t* qrow = qrow_of(col0 + gi);
        float qv[32];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 w4 = qrow ? reinterpret_cast<const uint4*>(qrow)[4 * ti + j] : make_uint4(0u, 0u, 0u, 0u);
          const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            qv[8 * j + 2 * i] = widen16(static_cast<uint16_t>(w[i] & 0xffff), a.dtype);
            qv[8 * j + 2 * i + 1] = widen16(static_cast<uint16_t>(w[i] >> 16), a.dtype);
          }
        }
        bool ok = true;
        float m = -INFINITY, l = 0.0f;
        const int pos_gi = SC ? pos_of(col0 + gi) : 0;
        const float slope_gi = SC ? ptile[gi * kPRow + kSlopeAt] : 0.0f;
        for (int i = 0; i < n; ++i) {
          const int s = i & 1;
          if (!((skip >> s) & 1u)) {
            if (!wait(s)) {
              ok = false;
              break;
            }
            const int u = u0 + i;   // a whole block
            kivi_block<FMT, SC>(a, reinterpret_cast<const char*>(s ? st1 : st0), ms, m, l, qv, a.sm_scale_log2,
                                SC ? pos_gi - (u < pl.A0 ? u : u + pl.F0 - pl.A0) * BT : 0, slope_gi);
          }
          if (i + kStages < n) issue(s, i + kStages);
        }
        mma_unscale<FMT>(ms);
        // into the cut blocks' form: maxima of columns 2ti, 2ti + 1 (the same in every
        // lane of a column), sums in lanes gi = 0
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        ms.m0 = __shfl_sync(0xffffffffu, m, 8 * ti);
        ms.m1 = __shfl_sync(0xffffffffu, m, 8 * ti + 4);
        const float l0 = __shfl_sync(0xffffffffu, l, 8 * ti), l1 = __shfl_sync(0xffffffffu, l, 8 * ti + 4);
        ms.l0 = lane < 4 ? l0 : 0.0f;
        ms.l1 = lane < 4 ? l1 : 0.0f;
        const int pos0 = pos_of(col0 + 2 * ti), pos1 = pos_of(col0 + 2 * ti + 1);
        for (int c = c0; ok && c < c1; ++c) {
          const int blk = pl.block_of(nf + c);
          const int t0 = kG * blk, t1 = min(t0 + kG, T);
          cut.tok0 = t0;
          const bool kquant = t0 + kG <= sg.Tk, vrec = t0 < sg.Tv;
          const bool kstaged = !kquant && !vrec && t1 - t0 <= kKringStageMax;
          const int np = t0 + kP < T ? 2 : 1;
          const int vt0 = max(t0, sg.Tv), nv = max(0, t1 - vt0);
          const int voff = kstaged ? (t1 - t0) * kD * 2 : kVoffRecsB<FMT>;
          int p0 = 0, p1 = 0;
          if (kquant || vrec) {
            p0 = page(2 * blk);
            p1 = np == 2 ? page(2 * blk + 1) : p0;
            if (p0 < 0 || p1 < 0) continue;
          }
          const uint32_t rb = vrec ? F::kBytes : F::kKm + 512;   // whole records, or the keys' part
          uint32_t bytes = nv * kD * 2;
          if (kquant || vrec) bytes += np * rb;
          if (kstaged) bytes += (t1 - t0) * kD * 2;
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) {
            mbar_expect_tx(&bar[0], bytes);
            if (kquant || vrec) {
              bulk_load_hint(st0, rec_at<FMT>(sg, p0), rb, &bar[0], once);
              if (np == 2) bulk_load_hint(st0 + RS, rec_at<FMT>(sg, p1), rb, &bar[0], once);
            }
            if (kstaged) bulk_load_hint(st0, kring, (t1 - t0) * kD * 2, &bar[0], once);
          }
          __syncwarp();
          if (lane < nv) {
            const int t = vt0 + lane;
            bulk_load_hint(st0 + voff + (t - t0) * kVRow, vring + static_cast<long long>(t % a.R) * kD, kD * 2, &bar[0], once);
          }
          pend |= 1u;
          if (!wait(0)) {
            ok = false;
            break;
          }
          kivi_cut_block<FMT, SC>(a, sg, ms, ptile, qv, reinterpret_cast<const char*>(st0),
                                  kstaged ? reinterpret_cast<const uint16_t*>(st0) : kring,
                                  reinterpret_cast<const char*>(st0 + voff), smem_u32(&zero16), a.sm_scale_log2,
                                  ptile + kSlopeAt, cut, pos0, pos1);
        }
        if (ok) {
          mma_to_gen(ms, gs, reinterpret_cast<float*>(st0));
          have = true;
        } else {
          fail(b);
        }
      }
      if (!have) gen_init(gs);
      const bool direct = !ONE && (own || !slot_ok);
      const int k = seg_start <= r0 ? 0 : 1;
      float* P = ONE ? reinterpret_cast<float*>(region) : a.ws + (2LL * gw + k) * partial_floats(a.pcols);
#pragma unroll
      for (int j = 0; j < kNH; ++j) {
        if (col0 + j < ncols && j < a.pcols) {
          if (direct) {
            const float l = gs.l[j], inv = l > 0.0f ? 1.0f / l : l == l ? 0.0f : l;
            store_out(a, out_row(col0 + j), lane, make_float4(gs.o[j][0] * inv, gs.o[j][1] * inv, gs.o[j][2] * inv, gs.o[j][3] * inv));
          } else {
            *reinterpret_cast<float4*>(P + j * kD + 4 * lane) = make_float4(gs.o[j][0], gs.o[j][1], gs.o[j][2], gs.o[j][3]);
            if (lane == 0) {
              (ONE ? one.wm[warp][j] : P[a.pcols * kD + 2 * j]) = gs.m[j];
              (ONE ? one.wl[warp][j] : P[a.pcols * kD + 2 * j + 1]) = gs.l[j];
            }
          }
        }
      }
      __syncwarp();   // the region is scratch until here
    }
    if (ONE) break;
    if (seg_start >= r0 && lane == 0) {   // this warp holds the segment's first unit: its merge descriptor
      int ncon = 0;
      if (!own && slot_ok) ncon = owner_of(seg_end - 1, C, n_act) - gw + 1;
      const long long first = 2LL * gw + (seg_start <= r0 ? 0 : 1);
      win_meta(a)[static_cast<long long>(b) * a.H * a.tiles + seg] =
          static_cast<long long>(static_cast<unsigned>(first)) | (static_cast<long long>(ncon) << 32);
    }
    // next segment
    seg_start = seg_end + kSegCost<FMT>;
    if (++seg == a.H * a.tiles) {
      seg = 0;
      if (++b >= a.B) break;
      T = a.seq_lens[b];
      pl = plan_of_warp<FMT, SC>(T, a, b, own_span);
    }
  }
  if (pend) fail(-1);   // never expected: every issued copy is waited for
  if constexpr (ONE) {
    const int h = seg / a.tiles, col0 = (seg - h * a.tiles) * NC;
    combine_cluster<FMT, NC, SC>(a, sm, one, static_cast<int>(gridDim.x), static_cast<int>(blockIdx.x), min(NC, ncols - col0),
                         static_cast<long long>(b) * a.nq * a.Hq + h * a.g, col0, a.g);
  }
}

// The contributors' partials of a split segment combined by the log-sum-exp rule,
// one output row an item. A warp takes kMC contributors at a time; with TEAM the
// four warps of a CTA share one row's contributors (a call of few segments: each
// has hundreds), otherwise each warp takes rows of its own.
template <bool TEAM>
__global__ void __launch_bounds__(32 * kMergeWarps) win_merge_kernel(DecodeArgs d, int tiles, int nc) {
  __shared__ float4 so[TEAM ? kMergeWarps : 1][32];
  __shared__ float sml[TEAM ? kMergeWarps : 1][2];
  asm volatile("griddepcontrol.wait;" ::: "memory");   // window_kernel has completed; its writes are visible
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long* desc = reinterpret_cast<const long long*>(d.ws + 2LL * d.grid_warps * partial_floats(d.pcols));
  const int ncols = d.nq * d.g;
  const long long items = static_cast<long long>(d.B) * d.H * ncols, pf = partial_floats(d.pcols);
  const long long it0 = TEAM ? blockIdx.x : static_cast<long long>(blockIdx.x) * kMergeWarps + warp;
  const long long step = TEAM ? gridDim.x : static_cast<long long>(gridDim.x) * kMergeWarps;
  constexpr int kShare = TEAM ? kMergeWarps : 1;   // warps of a row
  const int mine = TEAM ? warp : 0;
  for (long long it = it0; it < items; it += step) {
    const int col = static_cast<int>(it % ncols), tile = col / nc, j = col - tile * nc;
    const long long bh = it / ncols;
    const long long x = __ldcg(desc + bh * tiles + tile);
    const int n = static_cast<int>(x >> 32);
    if (n <= 0) continue;   // written by window_kernel
    const long long first = static_cast<long long>(static_cast<unsigned>(x & 0xffffffffLL));
    // contributor 0 is the descriptor's slot; i >= 1 is the warp i places on, slot 0
    auto part = [&](int i) -> const float* { return d.ws + (i == 0 ? first : (first & ~1LL) + 2LL * i) * pf; };
    float M = -INFINITY, L = 0.0f;
    float4 O = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int i0 = mine * kMC; i0 < n; i0 += kShare * kMC) {
      const int nch = min(kMC, n - i0);
      const float* W = part(i0 + (lane < nch ? lane : 0)) + d.pcols * kD + 2 * j;
      const float mi = lane < nch ? __ldcg(W) : -INFINITY;
      const float li = lane < nch ? __ldcg(W + 1) : 0.0f;
      float4 r[kMC];
#pragma unroll
      for (int u = 0; u < kMC; ++u)
        r[u] = u < nch ? __ldcg(reinterpret_cast<const float4*>(part(i0 + u) + j * kD + 4 * lane))
                       : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      const float mn = fmaxf(M, warp_max(mi));
      const bool live = mn != -INFINITY;   // every partial empty so far: nothing to weigh
      const float ao = live ? ex2(M - mn) : 1.0f, wi = live ? ex2(mi - mn) : 0.0f;
      L = fmaf(L, ao, warp_sum(wi * li));
      O = make_float4(O.x * ao, O.y * ao, O.z * ao, O.w * ao);
#pragma unroll
      for (int u = 0; u < kMC; ++u) {
        const float w = __shfl_sync(0xffffffffu, wi, u);
        if (u < nch) O = make_float4(fmaf(w, r[u].x, O.x), fmaf(w, r[u].y, O.y), fmaf(w, r[u].z, O.z), fmaf(w, r[u].w, O.w));
      }
      M = mn;
    }
    if constexpr (TEAM) {
      so[warp][lane] = O;
      if (lane == 0) {
        sml[warp][0] = M;
        sml[warp][1] = L;
      }
      __syncthreads();
      if (warp == 0) {
        float mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < kMergeWarps; ++w) mx = fmaxf(mx, sml[w][0]);
        L = 0.0f;
        O = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kMergeWarps; ++w) {
          const float l = sml[w][1];
          if (l == 0.0f) continue;
          const float f = mx == -INFINITY ? 1.0f : ex2(sml[w][0] - mx);
          const float4 y = so[w][lane];
          L = fmaf(f, l, L);
          O = make_float4(fmaf(f, y.x, O.x), fmaf(f, y.y, O.y), fmaf(f, y.z, O.z), fmaf(f, y.w, O.w));
        }
      }
      __syncthreads();
      if (warp != 0) continue;
    }
    const float inv = L > 0.0f ? 1.0f / L : L == L ? 0.0f : L;
    const int q = col / d.g;
    const long long row = (bh / d.H * d.nq + q) * d.Hq + (bh % d.H) * d.g + (col - q * d.g);
    store_out(d, row, lane, make_float4(O.x * inv, O.y * inv, O.z * inv, O.w * inv));
  }
}

// Grants a kernel its dynamic shared memory on the current device (once per device
// and size increase).
constexpr int kMaxDevices = 64;
std::mutex g_lock;
template <int FMT, int NC, bool ONE, bool SC>
cudaError_t grant(size_t need) {
  static size_t granted[kMaxDevices] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> guard(g_lock);
  if (need <= granted[dev]) return cudaSuccess;
  const void* f = reinterpret_cast<const void*>(window_kernel<FMT, NC, ONE, SC>);
  cudaError_t e = prefer_max_shared(f);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(need));
  if (e == cudaSuccess && ONE) e = cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) {
    cudaGetLastError();   // leave no error behind for the caller's next CUDA call
    return e;
  }
  granted[dev] = need;
  return cudaSuccess;
}
template <int FMT, int NC, bool SC> constexpr size_t kOneBytes = prefix_at<FMT, NC, SC>() + sizeof(OneSmem);
template <int FMT, int NC, bool SC>
cudaError_t one_ready() { return grant<FMT, NC, true, SC>(kOneBytes<FMT, NC, SC>); }

// A launch of `segs` clusters of `cluster` CTAs.
template <int FMT, int NC, bool SC>
void one_config(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr, int cluster, int segs, cudaStream_t st) {
  cfg->gridDim = dim3(static_cast<unsigned>(cluster), static_cast<unsigned>(segs));
  cfg->blockDim = dim3(32 * kWarps);
  cfg->dynamicSmemBytes = kOneBytes<FMT, NC, SC>;
  cfg->stream = st;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // as launch_behind
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg->attrs = attr;
  cfg->numAttrs = cluster > 1 ? 2 : 1;
}

// Clusters of `size` CTAs that the current device holds at once.
template <int FMT, int NC, bool SC>
int clusters_of(int size) {   // 2, 4, 8 or 16
  static int known_of[17][kMaxDevices] = {};   // 1 + the answer
  int(&known)[kMaxDevices] = known_of[size];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices || one_ready<FMT, NC, SC>() != cudaSuccess) return 0;
  std::lock_guard<std::mutex> guard(g_lock);
  if (known[dev] == 0) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    one_config<FMT, NC, SC>(&cfg, attr, size, 1, nullptr);
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, window_kernel<FMT, NC, true, SC>, &cfg) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    known[dev] = 1 + n;
  }
  return known[dev] - 1;
}

// Shape of a call: how many CTAs each segment takes in a launch that combines
// itself, 0 for the slices of the line and a combine kernel.
//
// A call of few segments is bound by latency, and the second kernel and the pass
// through the partials are much of it; a long one gains nothing from the fewer
// launches and loses where sequences differ in length, as a CTA's segment is its
// own. Measured (INT8, 8 kv heads, us, slices / clusters): 1 sequence of 2000
// tokens 10.6 / 8.2, of 32000 26.7 / 24.3; 16 of 2000 20.2 / 14.8; 32 of 1024 to
// 8192 tokens 54.5 / 63.6; 16 of 32000, all alike, 167.6 / 158.7, but the host knows
// only the longest. So: at most one segment per SM, and at most kOneTokens tokens per
// warp.
constexpr int kOneTokens = 384;
template <int FMT, int NC, bool SC>
int cluster_of(const WindowArgs& a, int num_sms) {
  const long long segs = static_cast<long long>(a.B) * a.H * a.tiles;
  if (a.form == 1 || segs > 65535 || (a.form == 0 && segs > num_sms)) return 0;
  const long long seen = static_cast<long long>(a.window) + a.nq + a.sinks;
  const long long blocks = (a.max_seq_len < seen ? a.max_seq_len : seen) / kBlock<FMT> + 2;   // of a segment, at most
  int c = 1;
  while (c < 8 && 2 * c * segs <= num_sms && blocks > static_cast<long long>(c) * kWarps) c *= 2;
  if (c == 8 && segs <= 6 && blocks > 16LL * kWarps) c = 16;   // (clusters of 16 fill a GPC each)
  // only what is resident at once: of 16 clusters of 8 some wait for a second pass (two sequences of 3000
  // tokens, 8 kv heads, one query: 4-bit 21.1 us, clusters of 4 12.2, slices 15.8; INT8 16.2, 10.9, 12.7)
  while (c > 1 && segs > clusters_of<FMT, NC, SC>(c)) c /= 2;
  if (a.form == 0 && blocks * kBlock<FMT> > static_cast<long long>(c) * kWarps * kOneTokens) return 0;
  return c;
}

template <int FMT, int NC, bool SC>
cudaError_t run_call(const Args<SC>& a, int num_sms, cudaStream_t st) {
  if (const int cluster = cluster_of<FMT, NC, SC>(a, num_sms)) {
    const cudaError_t e = one_ready<FMT, NC, SC>();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    one_config<FMT, NC, SC>(&cfg, attr, cluster, a.B * a.H * a.tiles, st);
    return cudaLaunchKernelEx(&cfg, window_kernel<FMT, NC, true, SC>, a);
  }
  // No more CTAs than the work can use (slices go to one warp of every CTA first):
  // a sequence has at most the blocks of max_seq_len, or of window, queries and
  // sinks, and each end of a range may cut one more.
  int grid = num_sms;
  const long long seen = static_cast<long long>(a.window) + a.nq + a.sinks;
  long long units = (a.max_seq_len < seen ? a.max_seq_len : seen) / kBlock<FMT> + 5;
  if (!kByte<FMT>) units += static_cast<long long>(a.tail_cost - 1) * ((a.R + 2 * kG) / kG + 5);
  const long long segs = static_cast<long long>(a.B) * a.H * a.tiles;
  const long long warps = (units * segs + kLeastUnits<FMT> - 1) / kLeastUnits<FMT>;
  if (warps < grid) grid = static_cast<int>(warps);
  const size_t smem = prefix_at<FMT, NC, SC>() + static_cast<size_t>(a.B + 1) * sizeof(long long);
  cudaError_t e = grant<FMT, NC, false, SC>(smem);
  if (e != cudaSuccess) return e;
  e = launch_behind(window_kernel<FMT, NC, false, SC>, dim3(static_cast<unsigned>(grid)), dim3(32 * kWarps), smem, st, a);
  if (e != cudaSuccess) return e;
  // the combine, launched programmatically right behind
  const long long items = static_cast<long long>(a.B) * a.H * a.nq * a.g;
  const bool team = static_cast<long long>(grid) * kWarps > 16 * segs;   // more than 16 partials a segment
  void (*f)(DecodeArgs, int, int) = team ? win_merge_kernel<true> : win_merge_kernel<false>;
  long long blocks = team ? items : (items + kMergeWarps - 1) / kMergeWarps;
  if (blocks > 16LL * num_sms) blocks = 16LL * num_sms;
  e = prefer_max_shared(reinterpret_cast<const void*>(f));
  if (e != cudaSuccess) return e;
  return launch_behind(f, dim3(static_cast<unsigned>(blocks)), dim3(32 * kMergeWarps), 0, st, static_cast<const DecodeArgs&>(a),
                       a.tiles, NC);
}

// The call of either kind on its page format.
template <bool SC>
cudaError_t launch_any(const Args<SC>& a, int num_sms, cudaStream_t st) {
  const bool wide = window_cols(a.bits, a.nq * a.g) == 16;
  switch (a.bits) {
    case kI8: return wide ? run_call<kI8, 16, SC>(a, num_sms, st) : run_call<kI8, 8, SC>(a, num_sms, st);
    case 8: return wide ? run_call<8, 16, SC>(a, num_sms, st) : run_call<8, 8, SC>(a, num_sms, st);
    case 2: return run_call<2, 8, SC>(a, num_sms, st);
    default: return run_call<4, 8, SC>(a, num_sms, st);
  }
}

}  // namespace
}  // namespace s4kv
