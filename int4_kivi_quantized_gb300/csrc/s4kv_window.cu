// Attention within a window (s4kv_window_attention) and all attention on INT8 pages: the
// kernels of s4kv_window.cuh without a score form.

#include "s4kv_window.cuh"

namespace s4kv {

int window_warps_per_sm() { return kWarps; }
int window_cols(int bits, int cols) { return (bits == 8 || bits == kI8) && cols > 8 ? 16 : 8; }

cudaError_t launch_window(const WindowArgs& a, int num_sms, cudaStream_t st) { return launch_any<false>(a, num_sms, st); }

}  // namespace s4kv
