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
// shuffle, and a rescale of O (when a maximum rises by more than kLazy) is the row's own.
//
// Warps 0 .. 3 and 4 .. 7 are the rows of the two tiles, warp 8 fetches (a ring of five 32 KB
// buffers, keys and values in turn, one bulk copy each), warp 9 issues the MMAs: P V and the next
// Q K^T of one tile while the other tile's rows are at their exponentials. The tensor
// cores execute one thread's MMAs in the order of issue, so that the next scores overwrite P
// only when P V has read it.
//
// Few rows behind a long cache: the kv tiles of a CTA are split over `splits` CTAs, whose
// outputs a third launch combines.

#include "s4kv_prompt.cuh"
#include "s4kv_tcgen05.cuh"

#include <mutex>

namespace s4kv {
namespace {

constexpr int kLoadWarp = 8, kMmaWarp = 9;
constexpr int kThreads = 320;
constexpr int kBufs = 5;
constexpr float kLazyP = 8.0f;       // P up to 2^8 before its sum divides it: exact enough in f16, and rescales are rare
constexpr int kQBytes = 128 * kD * 2;
constexpr int kSmemBytes = 2 * kQBytes + kBufs * kTileBytes + 1024;
// tensor memory columns: S (and P) of tile s at 128 s, O at 256 + 128 s
constexpr uint32_t kTmemCols = 512;

// D[tmem] (+)= A[tmem] B: A is K-major f16 pairs, a row a lane.
__device__ __forceinline__ void umma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u)
      : "memory");
}
// Shared-memory descriptor of a 128-byte swizzled MN-major operand: rows of 64 elements of MN, the
// next 64 `lbo` bytes on, the next eight rows (of K) 1024 bytes on.
__device__ __forceinline__ uint64_t umma_desc_mn(uint32_t saddr, uint32_t lbo) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(kSw128) << 61);
}
constexpr uint32_t kIdescQK = umma_idesc(128, 128);
constexpr uint32_t kIdescPV = umma_idesc(128, 128) | (1u << 16);   // B is MN-major

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

// A row's output (y: 32 channels from c0 on).
__device__ __forceinline__ void store32(void* out, int dtype, long long row, int c0, const float (&y)[32]) {
  const long long idx = row * kD + c0;
  if (dtype == S4KV_F32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(out) + idx);
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
  } else {
    uint4* p = reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + idx);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint4 w;
      w.x = pack_in_dtype(y[8 * i], y[8 * i + 1], dtype);
      w.y = pack_in_dtype(y[8 * i + 2], y[8 * i + 3], dtype);
      w.z = pack_in_dtype(y[8 * i + 4], y[8 * i + 5], dtype);
      w.w = pack_in_dtype(y[8 * i + 6], y[8 * i + 7], dtype);
      p[i] = w;
    }
  }
}

__device__ __forceinline__ float* part_rows(const PromptArgs& a, long long item) { return a.part + item * (kQRows * kD); }
__device__ __forceinline__ float* part_ml(const PromptArgs& a, long long item) {
  return a.part + static_cast<long long>(a.q_tiles) * a.H * a.splits * (kQRows * kD) + item * (2 * kQRows);
}

// One row's scores of a kv tile, from S to log2 units.
struct RowScore {
  float mul;       // no cap: S to log2 units. cap: S to x / cap
  float cap2;      // cap log2(e)
  float slope2;    // slope log2(e)
};

template <bool CAP, bool SLOPE>
__device__ __forceinline__ void score_form(float (&x)[128], const RowScore& f, float rel) {
  if constexpr (CAP) {
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 128; ++i) top = fmaxf(top, fabsf(x[i]));
    // (a score that is NaN does not show in `top` and stays NaN in both forms)
    if (__all_sync(0xffffffffu, top * f.mul <= 1.0f)) {
      const float2 mul2 = make_float2(f.mul, f.mul), cap2 = make_float2(f.cap2, f.cap2);
#pragma unroll
      for (int i = 0; i < 128; i += 2) {
        const float2 u = __fmul2_rn(make_float2(x[i], x[i + 1]), mul2), w = __fmul2_rn(u, u);
        float2 p = make_float2(tanh_coef(6), tanh_coef(6));
#pragma unroll
        for (int k = 5; k >= 0; --k) p = __ffma2_rn(p, w, make_float2(tanh_coef(k), tanh_coef(k)));
        p = __fmul2_rn(__fmul2_rn(u, cap2), p);
        x[i] = p.x;
        x[i + 1] = p.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 128; ++i) x[i] = f.cap2 * tanh_any(x[i] * f.mul);
    }
  } else if constexpr (SLOPE) {
#pragma unroll
    for (int i = 0; i < 128; ++i) x[i] *= f.mul;
  }
  if constexpr (SLOPE) {   // rel: the query's position less the tile's first token
#pragma unroll
    for (int i = 0; i < 128; ++i) x[i] = fmaf(-f.slope2, fabsf(static_cast<float>(i) - rel), x[i]);
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
    sm.abort = 0;
    sm.lo = 0x7fffffff;
    sm.hi = -1;
  }
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  stream_wait();
  Place pl;
  // the last tiles of a sequence, whose rows see the most, start first
  const int where = find_tile<kThreads, true>(a, static_cast<int>(gridDim.x - 1 - blockIdx.x), pl);
  if (where != kFound) return;
  const int h = blockIdx.y, z = blockIdx.z, b = pl.b, g = a.g;
  const int cu0 = a.cu_q[b], m = a.cu_q[b + 1] - cu0, T = a.seq_lens[b], slot = a.slot_ids ? a.slot_ids[b] : b;
  int arg;
  const int why = refused(a, pl, m, T, slot, h, arg);
  if (why && tid == 0) report(a.status, S4KV_ERR_DEVICE, why, arg);
  const int row0 = pl.tile * kQRows;
  const int rows = static_cast<int>(min(static_cast<long long>(kQRows), static_cast<long long>(m) * g - row0));
  const int tiles = rows > 128 ? 2 : 1;
  // a row's token of the chunk; its row of q and out
  auto token_of = [&](int r) { return (row0 + r) / g; };
  auto out_row = [&](int r) -> long long {
    const int i = token_of(r);
    return (static_cast<long long>(cu0) + i) * a.Hq + h * g + (row0 + r - i * g);
  };

  // ---- what each row sees; the queries as f16 operands ----
  Span sp{0, 0x7fffffff};   // (rows past the last one: everything, so that they ask for no masks)
  int pos = 0;
  if (tid < kQRows && !why) {
    if (tid < rows) {
      const int i = token_of(tid);
      pos = T - m + i;
      sp = span_of(a.form, pos, T, static_cast<long long>(cu0) + i, b);
    }
    const bool range = tid < rows && sp.lo <= sp.hi;
    const int lo = __reduce_min_sync(0xffffffffu, range ? sp.lo : 0x7fffffff);
    const int hi = __reduce_max_sync(0xffffffffu, tid < rows ? sp.hi : -1);
    if (lane == 0) {
      atomicMin(&sm.lo, lo);
      atomicMax(&sm.hi, hi);
    }
    const int c = lane & 15;
#pragma unroll 4
    for (int k = 0; k < 16; ++k) {
      const int r = 32 * warp + 2 * k + (lane >> 4);
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (r < rows) v = reinterpret_cast<const uint4*>(a.q + out_row(r) * kD)[c];
      float down = 1.0f;
      if (a.dtype == S4KV_BF16) {
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) top = __vmaxu2(top, w[i] & 0x7fff7fffu);
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
        const int pw = query_power(max(top & 0xffffu, top >> 16));
        const float up = power_of_two(pw);
        down = power_of_two(-pw);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = pack_f16x2(__uint_as_float(w[i] << 16) * up, __uint_as_float(w[i] & 0xffff0000u) * up);
        v = make_uint4(w[0], w[1], w[2], w[3]);
      }
      *reinterpret_cast<uint4*>(q_tiles + (r >> 7) * kQBytes + sw128_off(r & 127, 8 * c, 128)) = v;
      if (c == 0) sm.up[r] = down;
    }
    fence_proxy_async();
  }
  if (warp == kLoadWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm.tmem)), "n"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  // kv tiles that some row sees: the sinks' [0, sa), then [jb, je)
  const int last = sm.hi;
  const int sa = why ? 0 : (min(a.form.sinks, last + 1) + kKvTile - 1) / kKvTile;
  const int jb = max(sa, sm.lo == 0x7fffffff ? sa : sm.lo / kKvTile), je = why || sm.lo == 0x7fffffff ? jb : last / kKvTile + 1;
  const int all = sa + max(0, je - jb);
  const int i0 = static_cast<int>(static_cast<long long>(all) * z / a.splits);
  const int cnt = static_cast<int>(static_cast<long long>(all) * (z + 1) / a.splits) - i0;
  auto kv_of = [&](int i) { return i0 + i < sa ? i0 + i : jb + (i0 + i - sa); };
  auto tile_at = [&](int i) { return (static_cast<long long>(pl.kv0) + kv_of(i)) * a.H + h; };

  volatile int* flag = &sm.abort;
  // Bounded: false, and the flag that ends every role's loop raised, when it runs out.
  auto wait = [&](uint64_t* bar, int parity) -> bool {
    if (a.wait_ns > 0 && mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = global_ns();
    for (unsigned it = 1; a.wait_ns > 0; ++it) {
      if (mbar_try_wait(bar, parity)) return true;
      if (*flag) return false;
      if ((it & 15u) == 0 && static_cast<long long>(global_ns() - t0) > a.wait_ns) break;
    }
    *flag = 1;
    return false;
  };

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
      for (int it = max(0, sent - kBufs); it < sent; ++it) mbar_wait(&sm.full[it % kBufs], (it / kBufs) & 1, kDrainNs);
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    if (lane == 0 && cnt > 0) {
      const uint32_t q_s = smem_u32(q_tiles), ring_s = smem_u32(ring);
      auto qk = [&](int s, int i) {
        const uint32_t k_s = ring_s + ((2 * i) % kBufs) * kTileBytes;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          umma_f16(tmem + 128 * s, umma_desc(q_s + s * kQBytes + (j >> 2) * 16384 + (j & 3) * 32, 1024, kSw128),
                   umma_desc(k_s + (j >> 2) * 16384 + (j & 3) * 32, 1024, kSw128), kIdescQK, j > 0);
        umma_commit(&sm.sfull[s]);
      };
      auto pv = [&](int s, int i) {
        const uint32_t v_s = ring_s + ((2 * i + 1) % kBufs) * kTileBytes;
#pragma unroll
        for (int j = 0; j < 8; ++j)   // 16 tokens: 8 columns of P, 16 rows of 128 bytes
          umma_f16_ta(tmem + 256 + 128 * s, tmem + 128 * s + 8 * j, umma_desc_mn(v_s + j * 2048, 16384), kIdescPV, i > 0 || j > 0);
        umma_commit(&sm.odone[s]);
      };
      bool ok = wait(&sm.full[0], 0);
      if (ok) {
        tc_fence_after();
        for (int s = 0; s < tiles; ++s) qk(s, 0);
        umma_commit(&sm.empty[0]);
      }
      for (int i = 0; ok && i < cnt; ++i) {
        const int vi = 2 * i + 1, ki = 2 * i + 2;
        ok = wait(&sm.full[vi % kBufs], (vi / kBufs) & 1);
        for (int s = 0; ok && s < tiles; ++s) {
          ok = wait(&sm.pfull[s], i & 1);
          if (!ok) break;
          tc_fence_after();
          pv(s, i);
          if (s == tiles - 1) umma_commit(&sm.empty[vi % kBufs]);
          if (i + 1 < cnt) {
            if (s == 0) ok = wait(&sm.full[ki % kBufs], (ki / kBufs) & 1);
            if (!ok) break;
            qk(s, i + 1);
            if (s == tiles - 1) umma_commit(&sm.empty[ki % kBufs]);
          }
        }
      }
      // no MMA is in flight when the CTA ends
      umma_commit(&sm.drain);
      mbar_wait(&sm.drain, 0, kDrainNs);
      if (!ok) report(a.status, S4KV_ERR_DEVICE_TIMEOUT, S4KV_DEV_TIMEOUT, b);
    }
    __syncwarp();
  } else if ((warp >> 2) < tiles) {
    const int s = warp >> 2;
    const uint32_t t_row = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t s_at = tmem + 128 * s + t_row, o_at = tmem + 256 + 128 * s + t_row;
    constexpr float kLog2e = 1.4426950408889634f;
    RowScore f;
    const float scale = a.sm_scale * sm.up[tid];
    f.mul = CAP ? scale / a.form.cap : scale * kLog2e;
    f.cap2 = CAP ? a.form.cap * kLog2e : 0.0f;
    f.slope2 = SLOPE ? a.form.slopes[h * g + (row0 + tid) % g] * kLog2e : 0.0f;
    float mx = -INFINITY, l = 0.0f;
    bool ok = true;
    for (int i = 0; i < cnt; ++i) {
      const int t0 = kv_of(i) * kKvTile;
      const uint4 wild = *reinterpret_cast<const uint4*>(a.bad + 4 * tile_at(i));
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
      score_form<CAP, SLOPE>(x, f, static_cast<float>(pos - t0));
      const bool whole = t0 + kKvTile - 1 <= sp.hi && (t0 >= sp.lo || t0 + kKvTile <= a.form.sinks) && (wild.x | wild.y | wild.z | wild.w) == 0;
      if (!__all_sync(0xffffffffu, whole)) {
        // bits of the tokens that the row sees, 32 at a time
        const uint32_t wilds[4] = {wild.x, wild.y, wild.z, wild.w};
        auto below = [](int n) -> uint32_t { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; };
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int t = t0 + 32 * k;
          // (hi may be the largest int)
          const uint32_t seen = below(sp.hi - t >= 31 ? 32 : sp.hi - t + 1) & (~below(sp.lo - t) | below(a.form.sinks - t));
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
      float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int j = 0; j < 128; j += 8)
#pragma unroll
        for (int e = 0; e < 4; ++e) t4[e] = fmaxf(t4[e], fmaxf(x[j + 2 * e], x[j + 2 * e + 1]));
      float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
      constexpr bool kRaw = !CAP && !SLOPE;   // x are still S
      if (kRaw) top *= f.mul;
      if (__any_sync(0xffffffffu, top > mx + kLazyP)) {
        const float mn = top > mx + kLazyP ? top : mx;
        const float al = mx == -INFINITY ? 0.0f : exp2_fast(mx - mn);   // (nothing so far: l and O are zeros)
        if (i > 0) {
          ok = __all_sync(0xffffffffu, wait(&sm.odone[s], (i - 1) & 1));
          if (!ok) break;
          tc_fence_after();
          const float by = mx == mn ? 1.0f : al;
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
      const float2 mul2 = make_float2(kRaw ? f.mul : 1.0f, kRaw ? f.mul : 1.0f), base2 = make_float2(-base, -base);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t w[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          float2 y = make_float2(x[64 * k + 2 * j], x[64 * k + 2 * j + 1]);
          y = kRaw ? __ffma2_rn(y, mul2, base2) : __fadd2_rn(y, base2);
          y = make_float2(exp2_fast(y.x), exp2_fast(y.y));
          sum[j & 1] = __fadd2_rn(sum[j & 1], y);
          w[j] = pack_f16x2(y.x, y.y);
        }
        tmem_st32(s_at + 32 * k, w);
      }
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
    const long long item = (static_cast<long long>(gridDim.x - 1 - blockIdx.x) * a.H + h) * a.splits + z;
    const float inv = a.splits > 1 ? 1.0f : l > 0.0f ? 1.0f / l : l == l ? 0.0f : l;
#pragma unroll 1
    for (int k = 0; k < 4; ++k) {
      uint32_t o[32];
      if (some) {
        tmem_ld32(o_at + 32 * k, o);
        tmem_wait_ld();
      }
      float y[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) y[j] = some ? __uint_as_float(o[j]) * inv : 0.0f;
      if (tid < rows) {
        if (a.splits == 1) store32(a.out, a.out_dtype, out_row(tid), 32 * k, y);
        else if (some) store32(part_rows(a, item), S4KV_F32, tid, 32 * k, y);
      }
    }
    if (a.splits > 1 && tid < rows) {
      float* ml = part_ml(a, item) + 2 * tid;
      ml[0] = some ? mx : -INFINITY;
      ml[1] = some ? l : 0.0f;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
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
  for (int k = 0; k < 4; ++k) {
    const int r = 32 * blockIdx.z + 4 * warp + k;
    const long long at = static_cast<long long>(pl.tile) * kQRows + r;
    if (at >= static_cast<long long>(m) * a.g) return;
    float mi = -INFINITY, li = 0.0f;
    if (lane < a.splits) {
      const float* ml = part_ml(a, item0 + lane) + 2 * r;
      mi = __ldcg(ml);
      li = __ldcg(ml + 1);
    }
    const float M = warp_max(mi);
    // a part that saw nothing has l = 0 (and may have no rows at all); one with a NaN keeps it
    const float w = li == 0.0f ? 0.0f : M == -INFINITY ? 1.0f : exp2_fast(mi - M);
    const float L = warp_sum(w * li);
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int s = 0; s < a.splits; ++s) {
      const float ws = __shfl_sync(0xffffffffu, w, s), ls = __shfl_sync(0xffffffffu, li, s);
      if (ls == 0.0f) continue;
      const float4 y = __ldcg(reinterpret_cast<const float4*>(part_rows(a, item0 + s) + r * kD) + lane);
      o = make_float4(fmaf(ws, y.x, o.x), fmaf(ws, y.y, o.y), fmaf(ws, y.z, o.z), fmaf(ws, y.w, o.w));
    }
    const float inv = L > 0.0f ? 1.0f / L : L == L ? 0.0f : L;
    o = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    const int i = static_cast<int>(at / a.g);
    const long long row = (static_cast<long long>(cu0) + i) * a.Hq + h * a.g + (at - static_cast<long long>(i) * a.g);
    if (a.out_dtype == S4KV_F32) {
      reinterpret_cast<float4*>(static_cast<float*>(a.out) + row * kD)[lane] = o;
    } else {
      reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row * kD)[lane] =
          make_uint2(pack_in_dtype(o.x, o.y, a.out_dtype), pack_in_dtype(o.z, o.w, a.out_dtype));
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
  const dim3 grid(static_cast<unsigned>(a.q_tiles), static_cast<unsigned>(a.H), static_cast<unsigned>(a.splits));
  e = launch_behind(prompt_kernel<CAP, SLOPE>, grid, dim3(kThreads), kSmemBytes, st, a);
  if (e != cudaSuccess || a.splits == 1) return e;
  e = prefer_max_shared(reinterpret_cast<const void*>(prompt_join_kernel));
  if (e != cudaSuccess) return e;
  return launch_behind(prompt_join_kernel, dim3(grid.x, grid.y, kQRows / 32), dim3(256), 0, st, a);
}

}  // namespace

cudaError_t launch_prompt(const PromptArgs& a, cudaStream_t st) {
  if (a.form.cap > 0.0f) return a.form.slopes ? run<true, true>(a, st) : run<true, false>(a, st);
  return a.form.slopes ? run<false, true>(a, st) : run<false, false>(a, st);
}

}  // namespace s4kv
