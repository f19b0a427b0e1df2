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

// tanh(x) = x P(x^2) for |x| <= 1, P the polynomial of least relative error on [0, 1] (a
// weighted least-squares fit, 5.0e-8 in exact arithmetic, 1.6e-7 evaluated in binary32).
__host__ __device__ constexpr float tanh_coef(int i) {
  constexpr float c[7] = {0.9999999403953552f, -0.33332839608192444f, 0.13325203955173492f, -0.05345702916383743f,
                          0.020289979875087738f, -0.006203378550708294f, 0.0010410223621875048f};
  return c[i];
}

namespace {

// bf16 queries enter the MMAs as f16. Their range is the wider one, so each column is
// taken at the power of two 2^k that brings its largest element to 2^14 .. 2^15: exact,
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

// tanh(x) of any x. Beyond |x| = 1 as (1 - e) / (1 + e) with e = exp(-2 |x|) <= 0.14, which
// loses nothing there; ex2 and the reciprocal are off by 2^-22 or so relative. A tanh.approx
// (2^-11 relative) would move a score near a cap of 50 by 0.02.
__device__ __forceinline__ float tanh_any(float x) {
  const float w = x * x;
  float p = tanh_coef(6);
#pragma unroll
  for (int i = 5; i >= 0; --i) p = fmaf(p, w, tanh_coef(i));
  const float e = exp2_fast(fabsf(x) * -2.8853900817779268f);   // -2 log2(e)
  const float far = copysignf(__fdividef(1.0f - e, 1.0f + e), x);
  return fabsf(x) <= 1.0f ? x * p : far;                       // (NaN: far, which is NaN)
}

// The tokens that the query at position p of a sequence of T tokens sees; `at` is its place in
// `first`. No token at all where lo > hi (and no sink is that early).
struct Span {
  int lo, hi;
};
__device__ __forceinline__ Span span_of(const ScoreForm& f, int p, int T, long long at, int b) {
  Span s;
  s.lo = max(0, p - f.window + 1);
  if (f.first) s.lo = max(s.lo, f.first[at]);
  s.hi = p;
  if (f.prefix) s.hi = min(max(p, min(f.prefix[b], T) - 1), T - 1);
  return s;
}
__device__ __forceinline__ bool sees(const Span& s, int t, int sinks) { return t <= s.hi && (t >= s.lo || t < sinks); }

}  // namespace
}  // namespace s4kv
