// Attention with a score form (s4kv_scores): scores capped by a tanh, a bias that depends on
// distance, and each query's own range of visible tokens (window, document, prefix). What the
// kernels of short chunks (s4kv_window.cuh) and of prompts (s4kv_prompt.cu) share.
//
//   x = sm_scale q . k_t;  z_t = cap tanh(x / cap) - slope_j |p - t|
//   t is visible when t <= hi and (t >= lo or t < sinks)
//   lo = max(p - window + 1, first[query]), hi = min(max(p, prefix[sequence] - 1), T - 1)
#pragma once

#include "s4kv_common.cuh"

namespace s4kv {

// s4kv_scores with its arguments checked. cap 0: scores as they are; null pointers: no such part.
struct ScoreForm {
  const float* slopes;      // [Hq]
  const int* first;         // by query token
  const int* prefix;        // by sequence
  float cap;
  int window, sinks;        // window kNoWindow: none
};
constexpr int kNoWindow = 1 << 30;   // wider than any sequence

// Attention of the newest tokens with a score form (s4kv_score_attention).
struct ScoredArgs : WindowArgs {
  ScoreForm score;
  float cap2, icap2;        // cap log2(e) and its inverse; 0: no cap
};
cudaError_t launch_scored(const ScoredArgs& a, int num_sms, cudaStream_t st);

// Capping scores, x the score by the cap. Those of a model that was trained with a cap lie well within it: for |x| <= kNearCap
// tanh(x) = x P(x^2), P the cubic of least relative error there (a weighted least-squares fit,
// 5.5e-7). Beyond, tanh(x) = 1 - 2 / (1 + exp(2 x)), whose exponential and reciprocal are off by
// 2^-22 or so relative: 2^-22 of the cap in a score, for scores of half of it and more (and what
// shares a warp's step with them). tanh.approx (2^-11 relative) would move a score of 50 by 0.02.
constexpr float kNearCap = 0.5f;
constexpr int kNearCoefs = 4;
__host__ __device__ constexpr float near_coef(int i) {
  constexpr float c[kNearCoefs] = {0.999999463558197f, -0.33326318860054016f, 0.13190296292304993f, -0.04440222680568695f};
  return c[i];
}

namespace {

// bf16 queries enter the MMAs as f16 (s4kv_window.cuh). Their range is the wider one, so each column
// is taken at the power of two 2^k that brings its largest element to 2^14 .. 2^15: exact,
// and elements down to 2^-28 of the largest keep every bit. k of a column whose largest
// magnitude has the bits `top` (0 for zeros, infinities and NaN, which stay what they are).
__device__ __forceinline__ int query_power(uint32_t top) {
  const int e = static_cast<int>(top >> 7);
  return top == 0 || e == 255 ? 0 : min(14 + 127 - e, 120);
}
__device__ __forceinline__ float power_of_two(int k) { return __int_as_float((k + 127) << 23); }   // -126 <= k <= 127

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// cap tanh(x) of any x: `by` times the score is 2 x log2(e). NaN stays NaN.
__device__ __forceinline__ float far_cap(float score, float by, float cap) { return fmaf(-2.0f * cap, rcp_fast(1.0f + exp2_fast(score * by)), cap); }

// The tokens that the query at position p of a sequence of T tokens sees; `at` is its place in
// `first`. No token at all where lo > hi (and no sink is that early).
struct Span {
  int lo, hi;
};
// EARLY: read past the first cache, by a kernel that may look while a launch before it still runs.
template <bool EARLY = false>
__device__ __forceinline__ Span span_of(const ScoreForm& f, int p, int T, long long at, int b) {
  auto look = [](const int* x) { return EARLY ? __ldcg(x) : *x; };
  Span s;
  s.lo = max(0, p - f.window + 1);
  if (f.first) s.lo = max(s.lo, look(f.first + at));
  s.hi = p;
  if (f.prefix) s.hi = min(max(p, min(max(look(f.prefix + b), 0), T) - 1), T - 1);
  return s;
}
__device__ __forceinline__ bool sees(const Span& s, int t, int sinks) { return t <= s.hi && (t >= s.lo || t < sinks); }

}  // namespace
}  // namespace s4kv
