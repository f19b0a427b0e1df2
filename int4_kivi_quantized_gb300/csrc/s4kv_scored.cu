// Attention of the newest tokens with a score form (s4kv_score_attention): the kernels of
// s4kv_window.cuh with one.

#include "s4kv_window.cuh"

namespace s4kv {

cudaError_t launch_scored(const ScoredArgs& a, int num_sms, cudaStream_t st) { return launch_any<true>(a, num_sms, st); }

}  // namespace s4kv
