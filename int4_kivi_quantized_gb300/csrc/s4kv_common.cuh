// Internal definitions shared by the s4kv CUDA translation units (not part of
// the public ABI; see include/s4kv.h for the format and the calls).
#pragma once

#include <cuda_runtime.h>
#include <cuda_fp16.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include <mutex>

#include "../../include/s4kv.h"

namespace s4kv {

// Fixed geometry of the one supported configuration.
constexpr int kD = 128;          // head_dim
constexpr int kP = 16;           // tokens per page
constexpr int kG = 32;           // tokens per key group
constexpr int kGv = 32;          // channels per value group
// Record of one (page, kv head): key codes, key scale/min, value codes, value
// scale/min (fp32). 4-bit codes: 3072 bytes; 2-bit codes: 2048 bytes.
template <int BITS>
struct Rec {
  static_assert(BITS == 4 || BITS == 2, "4-bit or 2-bit codes");
  static constexpr int kBytes = BITS == 4 ? 3072 : 2048;
  static constexpr int kKc = 0;
  static constexpr int kKm = 256 * BITS;              // key codes: 16 tokens x 128 channels x BITS bits
  static constexpr int kVc = kKm + 512;
  static constexpr int kVm = kVc + 256 * BITS;
  static constexpr int kLevels = (1 << BITS) - 1;     // largest code
  static_assert(kVm + 512 == kBytes, "four regions fill the record");
};
// FP8 E4M3 record (bits = 8): 4096 bytes, key bytes then value bytes, one e4m3
// byte per element and no per-group metadata (one scale per layer, kv head and
// tensor, kept in the pool header).
template <>
struct Rec<8> {
  static constexpr int kBytes = 4096;
  static constexpr int kKc = 0;
  static constexpr int kVc = 2048;
};
// INT8 block record (bits = S4KV_BITS_INT8): key codes, value codes (one byte
// each), the block's key and value scale. 4128 bytes is whole 32-byte sectors.
template <>
struct Rec<S4KV_BITS_INT8> {
  static constexpr int kBytes = 4128;
  static constexpr int kKc = 0;
  static constexpr int kVc = 2048;
  static constexpr int kKs = 4096;
  static constexpr int kVs = 4100;
  static constexpr int kCopy = 4112;   // bytes that hold something, whole 16-byte units
};
constexpr int kRec = Rec<4>::kBytes;
constexpr int kKc = Rec<4>::kKc, kKm = Rec<4>::kKm, kVc = Rec<4>::kVc, kVm = Rec<4>::kVm;
inline int rec_bytes(int bits) {
  return bits == 2                ? Rec<2>::kBytes
         : bits == 8              ? Rec<8>::kBytes
         : bits == S4KV_BITS_INT8 ? Rec<S4KV_BITS_INT8>::kBytes
                                  : Rec<4>::kBytes;
}
constexpr int kMaxGroup = 8;     // largest GQA group (query heads per kv head)

// Status area at the start of the pool (int32 words): the first error, and the
// grid barrier of the decode step (arrival count, generation).
enum { ST_CODE = 0, ST_DETAIL = 1, ST_ARG = 2, ST_BAR_COUNT = 16, ST_BAR_GEN = 17 };

}  // namespace s4kv

struct s4kv_cache {
  s4kv_config cfg;
  char* pool;
  size_t pool_bytes;
  s4kv_layout lay;
  size_t counters_offset;   // int32 [max_slots][H_kv], reserved (no kernel uses it)
  int elem_bytes;
  int decode_warps;         // 0 = every warp of the grid
  int tail_cost;            // cost of a tail chunk in the decode work partition
  int decode_impl;          // 0 tensor-core, 1 FFMA
  int key_split;            // S4KV_OPT_KEY_SPLIT
  int mq_kernel;            // S4KV_OPT_MQ_KERNEL
  int window_form;          // S4KV_OPT_WINDOW_FORM
  int bits;                 // page format: 4, 2, 8 (FP8 E4M3) or S4KV_BITS_INT8
  long long wait_ns;
  int num_sms;
  int device;
};

namespace s4kv {

// Position rotation of an append (s4kv_append_rope); table null: none.
struct RopeArgs {
  const float* table;       // [max_pos][dim]: cosines, then sines
  const uint16_t* q;        // queries to turn, or null
  uint16_t* q_out;
  int max_pos, dim, interleaved, Hq;
};

struct AppendArgs {
  char* pages;              // layer page region
  char* kring;              // layer key ring region
  char* vring;              // layer value ring region
  int* lens;                // [max_slots][H] stored lengths of this layer
  int* status;
  const uint16_t* k;
  const uint16_t* v;
  const int* cu_new;
  const int* slot_ids;
  const int* seq_lens_before;
  const int* block_table;
  long long kring_slot, kring_head;   // element strides
  long long vring_slot, vring_head;
  int bt_stride, n, num_new, H, R, num_pages, max_slots, dtype;
  int bits;                 // code width: 4, 2 or 8 (FP8), or S4KV_BITS_INT8
  const float* fp8_scale;   // FP8: this layer's scales, key [H] then value [H]
  RopeArgs rope;
  int num_sms;
  int query_ctas;           // 8-bit pages: the grid's last CTAs, which turn queries and nothing else
  int dslot, dhead, each;   // the other CTAs' warps / H and % H, and the page slots over the former
  int step;                 // INT8 pages, decode step: one row per sequence, seq_lens_before holds the
  int max_len;              // lengths after it, each at most max_len
};

// Restore of token ranges (s4kv_gather) and, for INT8 pages, of one slot.
struct GatherArgs {
  const char* pages;
  const char* kring;
  const char* vring;
  const int* lens;
  int* status;
  const int* block_table;
  const int* seq_lens;
  const int* slot_ids;
  const int* first;         // or null: 0
  const int* cu_rows;
  void* out_k;
  void* out_v;
  const float* fp8_scale;
  long long kring_slot, kring_head, vring_slot, vring_head;
  int bt_stride, n, num_rows, H, R, num_pages, max_slots, dtype, out_dtype, bits;
};

struct DequantArgs {
  const char* pages;
  const char* kring;
  const char* vring;
  const int* lens;
  int* status;
  const int* bt_row;
  float* out_k;
  float* out_v;
  long long kring_slot, kring_head, vring_slot, vring_head;
  int slot, T, H, R, num_pages, max_slots, dtype;
  int bits;                 // code width: 4, 2 or 8 (FP8)
  const float* fp8_scale;   // FP8: this layer's scales, key [H] then value [H]
};

struct DecodeArgs {
  const char* pages;
  const char* kring;
  const char* vring;
  const int* lens;          // [max_slots][H] stored lengths of this layer
  int* status;
  const uint16_t* q;
  const int* block_table;
  const int* seq_lens;
  const int* slot_ids;
  void* out;
  float* ws;                // two partials per warp, then the partition record
  long long kring_slot, kring_head, vring_slot, vring_head;
  long long wait_ns;
  float sm_scale_log2;      // sm_scale * log2(e)
  int bt_stride, B, Hq, H, g, R, num_pages, max_slots, dtype, out_dtype;
  int max_warps;            // 0: every warp of the grid
  int tail_cost;            // work-partition cost of a tail chunk (key group = 1)
  int max_seq_len;
  int grid_warps;           // worker warps of the launch grid (sizes the partial area)
  int nq;                   // query tokens per sequence (multi-query path; 1 for decode)
  int tw;                   // warps per team (multi-query path): ceil(nq g / 8)
  int pcols;                // columns of one partial in the workspace: g (decode), 8 (multi-query)
  int key_split;            // decode main loop: low f16 part of q' on wide-scale key slices
  int mq_kernel;            // multi-query kernel choice (S4KV_OPT_MQ_KERNEL)
  int bits;                 // code width: 4, 2 or 8 (FP8)
  const float* fp8_scale;   // FP8: this layer's scales, key [H] then value [H]
  // decode step (s4kv_decode_step): the new key and value rows [B][H][128] of
  // the token each sequence appends before attending; null for attention only
  const uint16_t* knew;
  const uint16_t* vnew;
  int* lens_w;              // the stored lengths, written by the step
  unsigned* gbar;           // grid barrier words (arrivals, generation)
};

// Attention within a window (s4kv_window_attention), and every attention call on
// INT8 pages (window wider than any sequence, no sinks).
struct WindowArgs : DecodeArgs {
  int window, sinks;        // token t is visible at position p: t <= p, t > p - window or t < sinks
  int tiles;                // column tiles of a (sequence, kv head): nq g columns, pcols each
  int form;                 // S4KV_OPT_WINDOW_FORM
};

// Asks for the largest shared-memory carve-out for `func`, once per device and
// kernel: every kernel of the library then runs with the same L1/shared split, so
// an SM needs no reconfiguration between back-to-back launches of different
// kernels (decode, merge, append).
inline cudaError_t prefer_max_shared(const void* func) {
  constexpr int kMax = 256;
  static std::mutex lock;
  static int dev_of[kMax];
  static const void* fn_of[kMax];
  static int n = 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return cudaErrorInvalidDevice;
  }
  std::lock_guard<std::mutex> guard(lock);
  for (int i = 0; i < n; ++i)
    if (dev_of[i] == dev && fn_of[i] == func) return cudaSuccess;
  const cudaError_t e =
      cudaFuncSetAttribute(func, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return e;
  }
  if (n < kMax) {
    dev_of[n] = dev;
    fn_of[n] = func;
    ++n;
  }
  return cudaSuccess;
}

// Launches `f` so that its start-up overlaps the end of the work before it in the
// stream: the kernel waits on the device (stream_wait) before it touches memory.
template <typename... P, typename... A>
inline cudaError_t launch_behind(void (*f)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, f, static_cast<P>(args)...);
}
__device__ __forceinline__ void stream_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Host-side launchers (one per translation unit).
cudaError_t launch_append(const AppendArgs& a, int grid, cudaStream_t st);
int append_ctas_per_sm();   // resident CTAs per SM the append kernel is sized for
cudaError_t launch_dequant(const DequantArgs& a, cudaStream_t st);
cudaError_t launch_append8(const AppendArgs& a, int num_sms, cudaStream_t st);
cudaError_t launch_dequant_int8(const DequantArgs& a, cudaStream_t st);
cudaError_t launch_gather(const GatherArgs& a, int num_sms, cudaStream_t st);
cudaError_t launch_window(const WindowArgs& a, int num_sms, cudaStream_t st);
int window_cols(int bits, int cols);      // columns of one warp's tile for a call of `cols` columns
int window_warps_per_sm();
cudaError_t launch_decode(const DecodeArgs& a, int impl, int grid, cudaStream_t st);
// the decode step: a cooperative launch of the decode kernel with the append phase
cudaError_t launch_decode_step(const DecodeArgs& a, int impl, int grid, cudaStream_t st);
cudaError_t launch_mq(const DecodeArgs& a, int grid, cudaStream_t st);
int decode_threads(int impl);
int decode_warps_per_cta(int impl);
size_t decode_partial_bytes(int g);
size_t decode_meta_bytes(int B, int H);   // merge descriptors, one per (sequence, kv head)
size_t decode_trace_bytes_per_warp();   // 0 unless built with -DS4KV_DECODE_TRACE
size_t decode_smem_bytes(int impl, int B);
int decode_ctas_per_sm(int impl, int B);

// ---- device helpers ----------------------------------------------------------
__device__ __forceinline__ void report(int* status, int code, int detail, int arg) {
  if (atomicCAS(status + ST_CODE, 0, code) == 0) {
    status[ST_DETAIL] = detail;
    status[ST_ARG] = arg;
  }
}

// The stored length of a slot under an append of several work items (a (sequence, kv head)
// that had T0 tokens, T0 > 0, and gets T1 - T0 more). Each item looks whether the slot
// held T0 tokens when the launch began (goes_on) before it stores anything, and says so
// when it has looked (looked; once for a run of items, with their number `part` of
// `total`). The length changes while other items have still to look, so the word itself
// counts: the first turns T0 into minus its part, the others subtract theirs, the last one
// leaves T1. So a length that is T1 already (the same append again) is not taken for one
// that this launch made, and all items of a (sequence, head) decide alike.
__device__ __forceinline__ bool went_on(int v, int T0) { return v == T0 || v < 0; }
__device__ __forceinline__ bool goes_on(const int* len, int T0) { return went_on(__ldcg(len), T0); }
__device__ __forceinline__ void looked(int* len, int T0, int T1, int part, int total) {
  if (atomicCAS(len, T0, part < total ? -part : T1) != T0 && atomicAdd(len, -part) == part - total) atomicExch(len, T1);
}

__device__ __forceinline__ float widen16(uint16_t bits, int dtype) {
  if (dtype == S4KV_BF16) return __uint_as_float(static_cast<uint32_t>(bits) << 16);
  return __half2float(__ushort_as_half(bits));
}

__device__ __forceinline__ unsigned long long global_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

}  // namespace s4kv
